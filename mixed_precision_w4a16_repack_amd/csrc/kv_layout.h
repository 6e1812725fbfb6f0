// kv_layout.h -- where the elements of a paged key/value cache lie (defined
// in include/w4a16.h): shared by the writer, the reader and the attention.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

namespace w4a16 {

// Byte offsets inside one head's record of a page. KIND 0: 16-bit values,
// 1: int8 codes with a scale per token. Keys are tiles of 16 tokens, values
// tiles of 32 tokens, 1024 bytes each.
template <int KIND>
struct KvPlace {
    // Tile dimensions along d.
    static constexpr int kKeyD = KIND == 0 ? 32 : 64;
    static constexpr int kValD = KIND == 0 ? 16 : 32;

    static __device__ __forceinline__ int64_t key(int t, int d, int D) {
        const int64_t tile = (int64_t)(t / 16) * (D / kKeyD) + d / kKeyD;
        const int lane = d % 32 / 8 * 16 + t % 16;
        return tile * 1024 + lane * 16 + (KIND == 0 ? d % 8 * 2 : d % 64 / 32 * 8 + d % 8);
    }
    static __device__ __forceinline__ int64_t value(int t, int d, int D, int P) {
        const int64_t tile = (int64_t)(t / 32) * (D / kValD) + d / kValD;
        const int lane = t % 16 / 4 * 16 + d % 16;
        const int pos = t % 32 / 16 * 4 + t % 4;
        return keys_bytes(D, P) + tile * 1024 + lane * 16 + (KIND == 0 ? pos * 2 : d % 32 / 16 * 8 + pos);
    }
    static __host__ __device__ __forceinline__ int64_t keys_bytes(int D, int P) { return (int64_t)P * D * (KIND == 0 ? 2 : 1); }
    // int8 only: the scale of token t's key (0) or value (1).
    static __device__ __forceinline__ int64_t scale(int t, int D, int P, int which) {
        return 2 * keys_bytes(D, P) + (int64_t)(which * P + t) * 4;
    }
    static __host__ __device__ __forceinline__ int64_t record_bytes(int D, int P) {
        return 2 * keys_bytes(D, P) + (KIND == 0 ? 0 : (int64_t)P * 8);
    }
};

}  // namespace w4a16
