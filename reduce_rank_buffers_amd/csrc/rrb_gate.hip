// The gate of an MoE layer: from scores [tokens][experts], each token's top-k
// experts and their softmax weights, as rrb_moe_route takes them, and the
// gradient of the scores.
//
// One wave per token.  The experts are chosen on the scores themselves (the
// softmax keeps their order, and rounding a probability could only merge
// two), as a 64-bit key (score as an ordered integer, then the lower expert
// first), so the choice is exact and ties are decided.  Weights are fp32:
// w_i = e^(l_i - m) / sum, over all experts, or over the chosen ones.
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

__device__ __forceinline__ float load_score(const float *p) { return *p; }
__device__ __forceinline__ float load_score(const uint16_t *p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store_score(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_score(uint16_t *p, float v) { *p = f32_to_bf16_rne(v); }

// Orders scores as unsigned integers: -inf lowest, both zeros equal, every
// NaN above +inf (so a row with a NaN has it among its experts and shows it
// in its weights).  Always above 0.
__device__ __forceinline__ uint32_t score_key(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t u = __float_as_uint(f == 0.f ? 0.f : f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// e^(l - m), where an expert masked out by -inf has no share (also where all
// are) and scores of +inf share equally.
__device__ __forceinline__ float share(float l, float m) {
  if (l == -INFINITY) return 0.f;
  return l == m ? 1.f : expf(l - m);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}

// V = scores per lane: expert e sits in lane e % 64.
template <typename T, int V>
__global__ void __launch_bounds__(256) gate_kernel(GateArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = blockIdx.x * 4ll + (threadIdx.x >> 6);
  if (t >= a.tokens) return;
  const T *row = static_cast<const T *>(a.logits) + t * a.experts;
  float l[V];
  uint64_t key[V];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < a.experts ? load_score(row + e) : -INFINITY;
    key[i] = e < a.experts ? static_cast<uint64_t>(score_key(l[i])) << 32 | (0xffffffffu - e) : 0;
    m = fmaxf(m, l[i]);
  }
  m = wave_max(m);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) sum += share(l[i], m);
  sum = wave_sum(sum);
  float mine = 0.f;
  int chosen = 0;
  for (int j = 0; j < a.topk; ++j) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) best = key[i] > best ? key[i] : best;
#pragma unroll
    for (int d = 32; d; d >>= 1) {
      const uint64_t o = __shfl_xor(best, d, 64);
      best = o > best ? o : best;
    }
    const int e = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
    float le = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] == best) {
        key[i] = 0;
        le = l[i];
      }
    le = __shfl(le, e & 63, 64);
    if (lane == j) {
      chosen = e;
      mine = share(le, m);
    }
  }
  if (a.renorm) sum = wave_sum(mine);
  if (lane < a.topk) {
    a.idx[t * a.topk + lane] = chosen;
    a.w[t * a.topk + lane] = sum == 0.f ? 0.f : mine / sum;
  }
}

// With p the softmax over all experts and c the chosen ones' sum of p_i dw_i:
//   dl_j = p_j (dw_j - c) for a chosen expert, -p_j c for the others;
// renormalised, with w over the chosen ones alone, dl_i = w_i (dw_i - sum w dw)
// for these and 0 for the others.  A masked expert takes no part: its dw is
// not used.  Indices outside the experts are passed over.
template <typename T, int V>
__global__ void __launch_bounds__(256) gate_backward_kernel(GateArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = blockIdx.x * 4ll + (threadIdx.x >> 6);
  if (t >= a.tokens) return;
  const T *row = static_cast<const T *>(a.logits) + t * a.experts;
  T *out = static_cast<T *>(a.dlogits) + t * a.experts;
  const int32_t mine = lane < a.topk ? a.idx[t * a.topk + lane] : -1;
  const float dwj = lane < a.topk ? a.dw[t * a.topk + lane] : 0.f;
  float l[V], dw[V];
  bool on[V];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < a.experts ? load_score(row + e) : -INFINITY;
    m = fmaxf(m, l[i]);
    dw[i] = 0.f;
    on[i] = false;
  }
  for (int j = 0; j < a.topk; ++j) {
    const int e = __shfl(mine, j, 64);
    const float d = __shfl(dwj, j, 64);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e == i * 64 + lane && l[i] != -INFINITY) {
        on[i] = true;
        dw[i] = d;
      }
  }
  m = wave_max(m);
  float sum = 0.f, dot = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    l[i] = share(l[i], m);
    if (!a.renorm || on[i]) sum += l[i];
    if (on[i]) dot += l[i] * dw[i];
  }
  sum = wave_sum(sum);
  dot = wave_sum(dot);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const float mean = sum == 0.f ? 0.f : dot / sum;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 64 + lane;
    if (e >= a.experts) continue;
    float d = on[i] ? dw[i] - mean : a.renorm ? 0.f : -mean;
    d = l[i] == 0.f ? 0.f : l[i] * inv * d;
    store_score(out + e, d);
  }
}

using GateFn = void (*)(GateArgs);

template <typename T>
GateFn gate_for(int experts, bool back) {
  const int v = (experts + 63) / 64;
#define RRB_PICK(n) \
  if (v <= n) return back ? gate_backward_kernel<T, n> : gate_kernel<T, n>;
  RRB_PICK(1) RRB_PICK(2) RRB_PICK(4) RRB_PICK(8) RRB_PICK(16)
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
  const int64_t blocks = (a.tokens + 3) / 4;
  if (blocks > 0x7fffffffLL) return fail(RRB_EUNSUPPORTED, "too many tokens for one launch");
  if (a.tokens == 0) return RRB_OK;
  if (!a.logits || !a.idx || (back ? !a.dw || !a.dlogits : !a.w)) return fail(RRB_EINVAL, "NULL array");
  const GateFn fn = dtype == RRB_F32 ? gate_for<float>(a.experts, back) : gate_for<uint16_t>(a.experts, back);
  hipLaunchKernelGGL(fn, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, static_cast<hipStream_t>(stream), a);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? RRB_OK : fail(RRB_EHIP, "gate launch: %s", hipGetErrorString(e));
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
