// Loads from memory straight to LDS, shared by the experts' kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace rrb {

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
template <typename EL>
__device__ __forceinline__ const EL *uniform(const EL *q) {
  const uint64_t v = reinterpret_cast<uint64_t>(q);
  const uint32_t lo = uniform(static_cast<int>(v)), hi = uniform(static_cast<int>(v >> 32));
  // As a global address: through a plain one the loads would be flat, which
  // wait with the LDS's.
  typedef __attribute__((address_space(1))) const EL *global;
  return (const EL *)(global)(static_cast<uint64_t>(hi) << 32 | lo);
}

// A buffer of `bytes` from `base`, as the loads take it: accesses outside it give
// zeros and touch no memory.
template <typename EL>
__device__ __forceinline__ u32x4_t descriptor(const EL *base, int bytes) {
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
// STREAM: what is read once (nt), not kept in the caches.
template <bool STREAM = false>
__device__ __forceinline__ void load_to_lds(u32x4_t d, int at, int voffset, int soffset) {
  if (STREAM)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
                 :
                 : "s"(uniform(at)), "v"(voffset), "s"(d), "s"(uniform(soffset))
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(uniform(at)), "v"(voffset), "s"(d), "s"(uniform(soffset))
                 : "memory");
}

}  // namespace rrb
