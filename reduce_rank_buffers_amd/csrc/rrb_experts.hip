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
// kernel (rrb_product.h) in three forms that differ in which side has the
// reduction index contiguous in memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "rrb_internal.h"
#include "rrb_kernels.h"
#include "rrb_product.h"

namespace rrb {
namespace {

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
  ProductArgs<uint16_t> p;  // offsets, rows, groups
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

int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }

// Bytes of the arrays that the sizes name.
struct Bytes {
  int64_t x, y, w, bias, offsets;
  explicit Bytes(const rrb_expert_spec &s)
      : x(s.rows * s.in * 2), y(s.rows * s.out * 2), w(s.groups * s.in * s.out * 2), bias(s.groups * s.out * 2),
        offsets((s.groups + 1ll) * 4) {}
};

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
  ProductArgs<uint16_t> p = base_args<uint16_t>(*spec, d_offsets);
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
  ProductArgs<uint16_t> p = base_args<uint16_t>(*spec, d_offsets);
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
  ProductArgs<uint16_t> p = base_args<uint16_t>(*spec, d_offsets);
  p.a[0] = dgate;
  p.a[1] = dup;
  p.lda = g.ldo;
  p.halves = 2;
  p.n = static_cast<int32_t>(spec->in);
  if (d_dx && spec->rows > 0) {
    ProductArgs<uint16_t> q = p;
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
  ProductArgs<uint16_t> p = base_args<uint16_t>(*spec, d_offsets);
  p.a[0] = p.a[1] = u16(d_dout);
  p.lda = spec->out;
  // Without an activation dZ is dY itself; rows that do not start on 16-byte
  // boundaries are copied into padded ones first.
  const bool copy = (d_dx || d_dw) && (act || spec->out % 8 || !aligned(d_dout, 16));
  if (d_dbias) {
    BiasGradArgs b;
    std::memset(static_cast<void *>(&b), 0, sizeof b);
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
    ProductArgs<uint16_t> q = p;
    q.b[0] = q.b[1] = u16(d_w);
    q.c[0] = u16(d_dx);
    q.ldb = q.ldc = spec->in;
    q.k = static_cast<int32_t>(spec->out);
    if ((st = launch_product<kGradX, false>(q, s)) != RRB_OK) return st;
  }
  if (d_dw) {
    ProductArgs<uint16_t> q = p;
    q.b[0] = q.b[1] = u16(d_x);
    q.c[0] = q.c[1] = u16(d_dw);
    q.ldb = q.ldc = spec->in;
    q.m = static_cast<int32_t>(spec->out);
    if ((st = launch_product<kGradW, false>(q, s)) != RRB_OK) return st;
  }
  return RRB_OK;
}

}  // extern "C"
