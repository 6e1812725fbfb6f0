// exchange.h -- cross-workgroup exchange of split-K partial sums, shared by
// the skinny and tiled kernels.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

#include "device_common.h"

namespace w4a16 {

// Cross-workgroup exchange of split-K partial sums. Every access carries the
// sc1 cache policy (write-through to, or read from, the agent-wide coherence
// point): stores are agent-scope relaxed atomic stores of 64 bits, which the
// compiler lowers to sc1 stores; loads are sc1 loads in inline assembly.
__device__ __forceinline__ void store_coherent(float* p, const floatx4& v) {
    uint64_t* q = reinterpret_cast<uint64_t*>(p);
    __hip_atomic_store(q, __builtin_bit_cast(uint64_t, __builtin_shufflevector(v, v, 0, 1)), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(q + 1, __builtin_bit_cast(uint64_t, __builtin_shufflevector(v, v, 2, 3)), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_coherent2(float* p, float x, float y) {
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, make_float2(x, y)), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
// Four coherent 16-byte loads and the wait for them, in one asm statement so
// that no compiler-inserted instruction can read the destination registers
// while the loads are in flight (the compiler does not track asm loads).
__device__ __forceinline__ void load_coherent4(const float* p0, const float* p1, const float* p2, const float* p3,
                                               floatx4& v0, floatx4& v1, floatx4& v2, floatx4& v3) {
    asm volatile(
        "global_load_dwordx4 %0, %4, off sc1\n\t"
        "global_load_dwordx4 %1, %5, off sc1\n\t"
        "global_load_dwordx4 %2, %6, off sc1\n\t"
        "global_load_dwordx4 %3, %7, off sc1\n\t"
        "s_waitcnt vmcnt(0)"
        : "=&v"(v0), "=&v"(v1), "=&v"(v2), "=&v"(v3)
        : "v"(p0), "v"(p1), "v"(p2), "v"(p3)
        : "memory");
}
// One coherent 16-byte read as two agent-scope atomic 64-bit loads (sc1),
// which the compiler tracks like ordinary loads: many can be in flight.
__device__ __forceinline__ floatx4 load_coherent(const float* p) {
    const uint64_t* q = reinterpret_cast<const uint64_t*>(p);
    const uint64_t lo = __hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint64_t hi = __hip_atomic_load(q + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const float2 a = __builtin_bit_cast(float2, lo), b = __builtin_bit_cast(float2, hi);
    return floatx4{a.x, a.y, b.x, b.y};
}
// Eight coherent 16-byte loads and eight of 8 bytes at two byte offsets from
// eight uniform bases, with the wait in the same asm statement (as above).
__device__ __forceinline__ void load_coherent8(const float* const (&p)[8], uint32_t off4, uint32_t off2, floatx4 (&v)[8],
                                               float2 (&w)[8]) {
    asm volatile(
        "global_load_dwordx4 %0, %16, %18 sc1\n\t"
        "global_load_dwordx4 %1, %16, %19 sc1\n\t"
        "global_load_dwordx4 %2, %16, %20 sc1\n\t"
        "global_load_dwordx4 %3, %16, %21 sc1\n\t"
        "global_load_dwordx4 %4, %16, %22 sc1\n\t"
        "global_load_dwordx4 %5, %16, %23 sc1\n\t"
        "global_load_dwordx4 %6, %16, %24 sc1\n\t"
        "global_load_dwordx4 %7, %16, %25 sc1\n\t"
        "global_load_dwordx2 %8, %17, %18 sc1\n\t"
        "global_load_dwordx2 %9, %17, %19 sc1\n\t"
        "global_load_dwordx2 %10, %17, %20 sc1\n\t"
        "global_load_dwordx2 %11, %17, %21 sc1\n\t"
        "global_load_dwordx2 %12, %17, %22 sc1\n\t"
        "global_load_dwordx2 %13, %17, %23 sc1\n\t"
        "global_load_dwordx2 %14, %17, %24 sc1\n\t"
        "global_load_dwordx2 %15, %17, %25 sc1\n\t"
        "s_waitcnt vmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7]),
          "=&v"(w[0]), "=&v"(w[1]), "=&v"(w[2]), "=&v"(w[3]), "=&v"(w[4]), "=&v"(w[5]), "=&v"(w[6]), "=&v"(w[7])
        : "v"(off4), "v"(off2), "s"(p[0]), "s"(p[1]), "s"(p[2]), "s"(p[3]), "s"(p[4]), "s"(p[5]), "s"(p[6]), "s"(p[7])
        : "memory");
}
// The first four of them only.
__device__ __forceinline__ void load_coherent8_half(const float* const (&p)[8], uint32_t off4, uint32_t off2,
                                                    floatx4 (&v)[8], float2 (&w)[8]) {
    asm volatile(
        "global_load_dwordx4 %0, %8, %10 sc1\n\t"
        "global_load_dwordx4 %1, %8, %11 sc1\n\t"
        "global_load_dwordx4 %2, %8, %12 sc1\n\t"
        "global_load_dwordx4 %3, %8, %13 sc1\n\t"
        "global_load_dwordx2 %4, %9, %10 sc1\n\t"
        "global_load_dwordx2 %5, %9, %11 sc1\n\t"
        "global_load_dwordx2 %6, %9, %12 sc1\n\t"
        "global_load_dwordx2 %7, %9, %13 sc1\n\t"
        "s_waitcnt vmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(w[0]), "=&v"(w[1]), "=&v"(w[2]), "=&v"(w[3])
        : "v"(off4), "v"(off2), "s"(p[0]), "s"(p[1]), "s"(p[2]), "s"(p[3])
        : "memory");
}
// Waits until every vector memory access this wave issued has completed
// (write-through stores: reached the coherence point).
__device__ __forceinline__ void wait_vector_memory() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

}  // namespace w4a16
