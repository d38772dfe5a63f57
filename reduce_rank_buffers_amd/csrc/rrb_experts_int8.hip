// The experts' products with rows and weights held in 8-bit integers, for
// serving: rows are quantised one by one (s = max |x| / 127, q = x / s to the
// nearest integer), weights once, channel by channel, by the same call, and
//   linear   Y = act((Q Wq^T) s sw + b) + R
//   gated    H = act((Q Gq^T) s sg) * ((Q Uq^T) s su)
// with sums in 32-bit integers, which are exact.
#include <hip/hip_runtime.h>

#include <cstring>

#include "rrb_internal.h"
#include "rrb_kernels.h"
#include "rrb_product.h"

namespace rrb {
namespace {

// Reduction lengths whose sums fit 32 bits whatever the integers: 128 * 128
// times at most 2^17 - 1.
constexpr int64_t kMaxDepth = (int64_t(1) << 17) - 1;

// ---- quantisation ---------------------------------------------------------------

struct QuantizeArgs {
  const void *x;
  const int32_t *offsets;  // rows first .. last of [groups + 1], or NULL: all
  int8_t *q;
  float *scale;
  int64_t rows;
  int32_t groups, width;
};

// x / s to the nearest integer, ties to even, exactly: the quotient's integer by
// a product, then its remainder, which fp32 holds (x - n s is a multiple of the
// smaller of the two's last places, and at most about s).  Scales near or below
// fp32's normal range are brought up first, and a quotient that a rounded-down
// scale of few bits makes larger than 127 is kept there.
__device__ __forceinline__ int nearest(float x, float s) {
  if (s < 0x1p-60f) x *= 0x1p80f, s *= 0x1p80f;
  float n = rintf(x * (1.f / s));
  const float r = __builtin_fmaf(-n, s, x), half = 0.5f * s;
  const bool odd = static_cast<int>(n) & 1;
  if (fabsf(r) > half || (fabsf(r) == half && odd)) n += r > 0.f ? 1.f : -1.f;
  return static_cast<int>(fminf(fmaxf(n, -127.f), 127.f));
}

// Eight consecutive elements as they lie in memory, and as fp32.  `have` of them
// exist; the others are 0.
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
  u32x4_t w;
  __device__ __forceinline__ void load(const uint16_t *src, int have) { w = load_chunk(src, have); }
  // A whole one that is read once: past the caches, in lines that the wave reads whole.
  __device__ __forceinline__ void stream(const uint16_t *src, bool there) {
    typedef u32x4_t unaligned __attribute__((aligned(2)));
    w = u32x4_t{0, 0, 0, 0};
    if (there) w = __builtin_nontemporal_load(reinterpret_cast<const unaligned *>(src));
  }
  __device__ __forceinline__ float at(int i) const { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }
  // The largest |x| as fp32 bits, two by two: bf16 patterns order as the values do.
  __device__ __forceinline__ uint32_t most(uint32_t than) const {
    typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
    u16x2_t m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t bits = w[i] & 0x7fff7fffu;
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, bits));
    }
    return max(than, static_cast<uint32_t>(max(m[0], m[1])) << 16);
  }
  // Keeps the row as it lies in memory until it is used again.
  __device__ __forceinline__ void keep() { asm volatile("" : "+v"(w)); }
};
template <>
struct Eight<float> {
  float w[8];
  __device__ __forceinline__ void load(const float *src, int have) {
    if (have >= 8) {
      __builtin_memcpy(w, src, sizeof w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = i < have ? src[i] : 0.f;
    }
  }
  __device__ __forceinline__ void stream(const float *src, bool there) { load(src, there ? 8 : 0); }
  __device__ __forceinline__ float at(int i) const { return w[i]; }
  __device__ __forceinline__ uint32_t most(uint32_t than) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) than = max(than, __float_as_uint(w[i]) & 0x7fffffffu);
    return than;
  }
  __device__ __forceinline__ void keep() {}
};

// L lanes (a wave's 64, or a workgroup's 256 or 1024) share a row, eight elements
// each by turns, the row's last eight where fewer are left (what two lanes have, both
// write alike).  HELD: at most so many turns, which stay in registers; 0: any width,
// the row read twice.  WHOLE: rows of at least eight.
template <typename T, int L, int HELD, bool WHOLE>
__global__ void __launch_bounds__(L == 64 ? 256 : L) quantize_kernel(QuantizeArgs a) {
  constexpr int ROWS = L == 64 ? 4 : 1;  // per workgroup at a time
  __shared__ uint32_t part[L / 64];
  const int lane = threadIdx.x & (L - 1);
  auto at = [&](int c) { return WHOLE ? min(c, a.width - 8) : c; };
  int64_t first = 0, last = a.rows;
  if (a.offsets) {
    first = a.offsets[0], last = a.offsets[a.groups];
    if (first < 0) first = 0;
    if (last > a.rows) last = a.rows;
  }
  for (int64_t row = first + blockIdx.x * static_cast<int64_t>(ROWS) + uniform(static_cast<int>(threadIdx.x / L));
       row < last; row += gridDim.x * static_cast<int64_t>(ROWS)) {
    const T *x = static_cast<const T *>(a.x) + row * a.width;
    int8_t *q = a.q + row * a.width;
    Eight<T> v[HELD ? HELD : 1];
    // The largest |x| as its bits, which order as the values do and put
    // infinities and NaN above them.
    uint32_t most = 0;
    if (HELD) {
#pragma unroll
      for (int h = 0; h < HELD; ++h) v[h].stream(x + at((h * L + lane) * 8), (h * L + lane) * 8 < a.width);
#pragma unroll
      for (int h = 0; h < HELD; ++h) {
        most = v[h].most(most);
        v[h].keep();
      }
    } else {
      for (int c = lane * 8; c < a.width; c += L * 8) {
        v[0].load(x + at(c), WHOLE ? 8 : a.width - c);
        most = v[0].most(most);
      }
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), d, 64)));
    if (L > 64) {
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = most;
      __syncthreads();
      for (int i = 0; i < L / 64; ++i) most = max(most, part[i]);
      __syncthreads();
    }
    most = uniform(static_cast<int>(most));
    const bool fine = most < 0x7f800000u;
    const float s = fine ? __uint_as_float(most) / 127.f : __uint_as_float(0x7fc00000u);
    if (lane == 0) a.scale[row] = s;
    // Rows of zeros, or with an infinity or a NaN, become zeros.
    const bool any = fine && s > 0.f;
    const bool small = s < 0x1p-100f;
    const float inv = any && !small ? 1.f / s : 0.f;
    // The integer as the last bits of a sum that has its unit in the last place;
    // where the quotient's error could decide, exactly.
    auto put = [&](int c, const Eight<T> &e, int have) {
      constexpr float kUnit = 12582912.f;  // 1.5 * 2^23
      uint32_t n[8];
      float far = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = __builtin_fmaf(e.at(i), inv, kUnit);
        far = fmaxf(far, fabsf(__builtin_fmaf(e.at(i), inv, kUnit - t)));
        n[i] = __float_as_uint(t);
      }
      if (any && (small || far > 0.5f - 0x1p-16f)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = static_cast<uint32_t>(nearest(e.at(i), s));
      }
      uint32_t w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t lo = (n[4 * i] & 255u) | (n[4 * i + 1] & 255u) << 8;
        const uint32_t hi = (n[4 * i + 2] & 255u) | (n[4 * i + 3] & 255u) << 8;
        w[i] = any ? lo | hi << 16 : 0u;
      }
      if (have >= 8) {
        __builtin_memcpy(q + c, w, 8);
      } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
          if (i < have) q[c + i] = static_cast<int8_t>(w[i >> 2] >> (8 * (i & 3)));
      }
    };
    if (HELD) {
#pragma unroll
      for (int h = 0; h < HELD; ++h)
        if ((h * L + lane) * 8 < a.width) put(at((h * L + lane) * 8), v[h], 8);
    } else {
      for (int c = lane * 8; c < a.width; c += L * 8) {
        v[0].load(x + at(c), WHOLE ? 8 : a.width - c);
        put(at(c), v[0], WHOLE ? 8 : a.width - c);
      }
    }
  }
}

// A wave per row where rows are many and at most 4096 wide, else a workgroup of 256,
// or of 1024 beyond 8192 (us: 8000 x 4096 bf16 28 by waves, 31 by 256 lanes; 4096 x
// 7168 30 and 26; 16 x 7168 10.6 and 5.6; 32768 x 7168 127 and 125, 5.5 TB/s, where
// loads that stay in the caches took 140 and rows held as fp32 163).
template <typename T>
void launch_quantize(const QuantizeArgs &a, hipStream_t s) {
  void (*kernel)(QuantizeArgs);
  const int lanes = a.width > 8192 ? 1024 : a.width > 512 && (a.rows < 4096 || a.width > 4096) ? 256 : 64;
  const int turns = (a.width + lanes * 8 - 1) / (lanes * 8);
  // (A row of 64 lanes takes at most eight turns, of 256 four, of 1024 two or more.)
  if (a.width < 8)
    kernel = quantize_kernel<T, 64, 0, false>;
  else if (lanes == 64)
    kernel = turns <= 1   ? quantize_kernel<T, 64, 1, true>
             : turns <= 2 ? quantize_kernel<T, 64, 2, true>
             : turns <= 4 ? quantize_kernel<T, 64, 4, true>
                          : quantize_kernel<T, 64, 8, true>;
  else if (lanes == 256)
    kernel = turns <= 1   ? quantize_kernel<T, 256, 1, true>
             : turns <= 2 ? quantize_kernel<T, 256, 2, true>
                          : quantize_kernel<T, 256, 4, true>;
  else
    kernel = turns <= 2   ? quantize_kernel<T, 1024, 2, true>
             : turns <= 4 ? quantize_kernel<T, 1024, 4, true>
             : turns <= 8 ? quantize_kernel<T, 1024, 8, true>
                          : quantize_kernel<T, 1024, 0, true>;
  const int rows = lanes == 64 ? 4 : 1;
  const int64_t blocks = (a.rows + rows - 1) / rows;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks < (1 << 20) ? blocks : 1 << 20)),
                     dim3(lanes == 64 ? 256 : lanes), 0, s, a);
}

// ---- the products -----------------------------------------------------------------

// Bytes of the arrays that the sizes name.
struct Bytes {
  int64_t x, xs, y, w, ws, bias, offsets;
  explicit Bytes(const rrb_expert_spec &s)
      : x(s.rows * s.in), xs(s.rows * 4), y(s.rows * s.out * 2), w(s.groups * s.in * s.out), ws(s.groups * s.out * 4),
        bias(s.groups * s.out * 2), offsets((s.groups + 1ll) * 4) {}
};

rrb_status check_int8(const rrb_expert_spec *s, const int32_t *offsets) {
  const rrb_status st = check_spec(s, offsets);
  if (st != RRB_OK) return st;
  if (s->in > kMaxDepth)
    return fail(RRB_EUNSUPPORTED, "in %lld: at most 2^17 - 1, so that sums fit 32 bits", (long long)s->in);
  return RRB_OK;
}

ProductArgs<int8_t> int8_args(const rrb_expert_spec &s, const int32_t *offsets) {
  ProductArgs<int8_t> p = base_args<int8_t>(s, offsets);
  p.lda = p.ldb = s.in;
  p.ldc = s.out;
  p.n = static_cast<int32_t>(s.out);
  p.k = static_cast<int32_t>(s.in);
  p.act = s.activation;
  return p;
}

}  // namespace
}  // namespace rrb

using namespace rrb;

extern "C" {

rrb_status rrb_quantize_rows(int64_t rows, int64_t width, int32_t dtype, const void *d_x, const int32_t *d_offsets,
                             int32_t groups, int8_t *d_q, float *d_scale, rrb_stream_t stream) {
  clear_error();
  if (rows < 0 || width < 1)
    return fail(RRB_EINVAL, "rows %lld, width %lld: rows >= 0, width >= 1 needed", (long long)rows, (long long)width);
  if (dtype != RRB_BF16 && dtype != RRB_F32) return fail(RRB_EINVAL, "unknown dtype %d", dtype);
  if (d_offsets && groups < 1) return fail(RRB_EINVAL, "offsets of %d groups", groups);
  if (rows >= 1LL << 31) return fail(RRB_EUNSUPPORTED, "rows %lld >= 2^31", (long long)rows);
  if (width > kMaxWidth) return fail(RRB_EUNSUPPORTED, "width %lld: at most 2^20", (long long)width);
  if (rows == 0) return RRB_OK;
  if (!d_x || !d_q || !d_scale) return fail(RRB_EINVAL, "NULL x, q or scale");
  const Span spans[] = {{d_x, rows * width * elem_size(dtype), "x", false},
                        {d_offsets, d_offsets ? (groups + 1ll) * 4 : 0, "offsets", false},
                        {d_q, rows * width, "q", true},
                        {d_scale, rows * 4, "scale", true}};
  const rrb_status st = check_disjoint(spans);
  if (st != RRB_OK) return st;
  const QuantizeArgs a = {d_x, d_offsets, d_q, d_scale, rows, groups, static_cast<int32_t>(width)};
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == RRB_BF16)
    launch_quantize<uint16_t>(a, s);
  else
    launch_quantize<float>(a, s);
  return launched("quantisation");
}

rrb_status rrb_expert_linear_int8(const rrb_expert_spec *spec, const int8_t *d_x, const float *d_x_scale,
                                  const int32_t *d_offsets, const int8_t *d_w, const float *d_w_scale,
                                  const void *d_bias, const void *d_residual, void *d_out, rrb_stream_t stream) {
  clear_error();
  rrb_status st = check_int8(spec, d_offsets);
  if (st != RRB_OK) return st;
  if (spec->rows == 0) return RRB_OK;
  if (!d_x || !d_x_scale || !d_w || !d_w_scale || !d_out)
    return fail(RRB_EINVAL, "NULL x, x_scale, w, w_scale or out");
  const Bytes z(*spec);
  // A tile's residual is read before any of the tile is written, and by no
  // other workgroup: it may be the output itself.
  const Span spans[] = {{d_x, z.x, "x", false}, {d_x_scale, z.xs, "x_scale", false},
                        {d_offsets, z.offsets, "offsets", false}, {d_w, z.w, "w", false},
                        {d_w_scale, z.ws, "w_scale", false}, {d_bias, z.bias, "bias", false},
                        {d_residual == d_out ? nullptr : d_residual, z.y, "residual", false},
                        {d_out, z.y, "out", true}};
  if ((st = check_disjoint(spans)) != RRB_OK) return st;
  ProductArgs<int8_t> p = int8_args(*spec, d_offsets);
  p.a[0] = p.a[1] = d_x;
  p.b[0] = p.b[1] = d_w;
  p.row = d_x_scale;
  p.col[0] = p.col[1] = d_w_scale;
  p.c[0] = u16(d_out);
  p.bias = u16(d_bias);
  p.residual = u16(d_residual);
  return launch_product<kForward, false>(p, static_cast<hipStream_t>(stream));
}

rrb_status rrb_expert_gated_int8(const rrb_expert_spec *spec, const int8_t *d_x, const float *d_x_scale,
                                 const int32_t *d_offsets, const int8_t *d_w_gate, const float *d_gate_scale,
                                 const int8_t *d_w_up, const float *d_up_scale, void *d_out, rrb_stream_t stream) {
  clear_error();
  rrb_status st = check_int8(spec, d_offsets);
  if (st != RRB_OK) return st;
  if (spec->rows == 0) return RRB_OK;
  if (!d_x || !d_x_scale || !d_w_gate || !d_gate_scale || !d_w_up || !d_up_scale || !d_out)
    return fail(RRB_EINVAL, "NULL x, w_gate, w_up, a scale or out");
  const Bytes z(*spec);
  const Span spans[] = {{d_x, z.x, "x", false}, {d_x_scale, z.xs, "x_scale", false},
                        {d_offsets, z.offsets, "offsets", false}, {d_w_gate, z.w, "w_gate", false},
                        {d_gate_scale, z.ws, "gate_scale", false}, {d_w_up, z.w, "w_up", false},
                        {d_up_scale, z.ws, "up_scale", false}, {d_out, z.y, "out", true}};
  if ((st = check_disjoint(spans)) != RRB_OK) return st;
  ProductArgs<int8_t> p = int8_args(*spec, d_offsets);
  p.a[0] = p.a[1] = d_x;
  p.b[0] = d_w_gate;
  p.b[1] = d_w_up;
  p.row = d_x_scale;
  p.col[0] = d_gate_scale;
  p.col[1] = d_up_scale;
  p.c[0] = u16(d_out);
  return launch_product<kForward, true>(p, static_cast<hipStream_t>(stream));
}

}  // extern "C"
