// attention_common.h -- device helpers of the attention kernels
// (attention.hip, attention_tokens.hip): probabilities as matrix operands,
// int8 codes as fp16 numbers, sums and reads across lanes.
#pragma once

#include "device_common.h"

namespace w4a16 {

constexpr float kLowest = -3.402823466e38f;

typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

// The factor on probabilities, and how far (in powers of 2) a score may pass
// the reference: in fp16 2^13 * 2^2 < 65504.
template <bool F16P>
struct Prob {
    static constexpr float kBias = F16P ? 13.0f : 0.0f;
    static constexpr float kHeadroom = F16P ? 2.0f : 8.0f;
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Maximum, or sum, over the four lane groups of a column (lanes l, l + 16, ...).
__device__ __forceinline__ float column_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float column_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Four int8 codes (one word) as two words of exact fp16 pairs.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t x = w ^ 0x80808080u;
    const half2_t off{(_Float16)-1152.0f, (_Float16)-1152.0f};
    const half2_t a = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, x, 0x04010400u)) + off;
    const half2_t b = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, x, 0x04030402u)) + off;
    lo = __builtin_bit_cast(uint32_t, a);
    hi = __builtin_bit_cast(uint32_t, b);
}
__device__ __forceinline__ u32x4 codes8_to_f16(uint32_t w0, uint32_t w1) {
    uint32_t a, b, c, d;
    codes_to_f16(w0, a, b);
    codes_to_f16(w1, c, d);
    return u32x4{a, b, c, d};
}

// A pointer that is the same on all lanes, in scalar registers.
__device__ __forceinline__ const float* uniform(const float* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v), hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
    return reinterpret_cast<const float*>((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ int64_t read_lane(int64_t v, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// v of the lane that a DPP control names, 0 where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t from_lane(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xF, false);
    return (int64_t)((uint64_t)hi << 32 | lo);
}
// Sum over lanes 0 .. lane.
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
    v += from_lane<0x111, 0xF>(v);  // row_shr:1, 2, 4, 8: within 16 lanes
    v += from_lane<0x112, 0xF>(v);
    v += from_lane<0x114, 0xF>(v);
    v += from_lane<0x118, 0xF>(v);
    v += from_lane<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
    v += from_lane<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
    return v;
}

// The loads before this are issued before anything after it.
__device__ __forceinline__ void issue_fence() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// a / b of non-negative numbers below 2^53 whose quotient is below 2^20: the
// product is off by less than 1 before it is cut.
__device__ __forceinline__ int divide(int64_t a, int64_t b) {
    const int q = (int)((double)a * __builtin_amdgcn_rcp((double)b));
    const int64_t r = a - q * b;
    return r < 0 ? q - 1 : (r >= b ? q + 1 : q);
}

// Two probabilities as NP packed operands, each what the ones before leave.
// fp16 is cut, not rounded (one instruction a pair), where a next operand takes
// what is cut off; a last one is rounded, two by one instruction (4 % of the time
// of long int8 trees, against one by one and packing).
template <int PDT, int NP>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&out)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        if constexpr (PDT == 0 && NP > 1) {
            const auto h = __builtin_amdgcn_cvt_pkrtz(x, y);
            out[i] = __builtin_bit_cast(uint32_t, h);
            x = __builtin_fmaf((float)h[0], -1.0f, x);
            y = __builtin_fmaf((float)h[1], -1.0f, y);
        } else if constexpr (PDT == 0) {  // both rounded by one instruction
            typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
            typedef float float2_t __attribute__((ext_vector_type(2)));
            out[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(float2_t{x, y}, half2_t));
        } else {
            typedef float float2_t __attribute__((ext_vector_type(2)));
            out[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(float2_t{x, y}, bf16x2_t));
            x -= __builtin_bit_cast(float, out[i] << 16);
            y -= __builtin_bit_cast(float, out[i] & 0xFFFF0000u);
        }
    }
}

}  // namespace w4a16
