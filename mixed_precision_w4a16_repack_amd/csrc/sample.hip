// sample.hip -- a token from each row of logits: temperature, top-k, top-p
// and min-p, from given uniform numbers (definition in include/w4a16.h).
//
// A 16-bit logit has at most 65536 values, so a row's sorted order is its
// histogram over them: one pass counts (one LDS atomic a logit, no exp), and
// everything after works on the values that occur. All tokens of a value have
// the same weight exp((x - max) / T), which is computed once a value in fp64,
// and each of top-k, top-p and min-p keeps a first part of the sorted order,
// so the kept set is a number of tokens, and the drawn one a place in the
// order: a value, and how many tokens of that value come before. A second pass
// finds that token by its index. Counts are whole numbers and sums are fp64 in
// a fixed order: nothing depends on the order of the atomics.
//
// One workgroup of 16 waves a row; 128 KB of LDS hold the counts, 16 bits each
// (kCarry of a value that is more frequent go to a list).
#include "device_common.h"
#include "internal.h"

namespace w4a16 {
namespace {

typedef u32x4 u32x4_any __attribute__((aligned(2)));

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kKeys = 1 << 16;
constexpr int kBlocks = kKeys / 64;  // of 64 values each, one a thread in the scan
constexpr uint32_t kCarry = 1u << 15;
constexpr int kCarries = (int)(kSampleMaxV / kCarry);
constexpr int kNone = -1;

// Order-preserving key of a logit's bits, 0 for one that is never drawn (-infinity,
// NaN); -0 counts as 0.
template <int DT>
__device__ __forceinline__ uint32_t key_of(uint32_t b) {
    constexpr uint32_t inf = DT == 0 ? 0x7C00u : 0x7F80u;
    const uint32_t mag = b & 0x7FFFu;
    if (mag > inf || b == (inf | 0x8000u)) return 0;
    if (mag == 0) return 0x8000u;
    return b & 0x8000u ? b ^ 0xFFFFu : b | 0x8000u;
}
template <int DT>
__device__ __forceinline__ float value_of(uint32_t key) {
    return act_to_float<DT>((uint16_t)(key & 0x8000u ? key & 0x7FFFu : key ^ 0xFFFFu));
}

// 2^t for t <= 0: e^(f ln 2) of the part below 1/2 as a Taylor sum (its rest is below 2^-47).
__device__ __forceinline__ double exp2_of(double t) {
    if (!(t > -1070.0)) return 0.0;
    const double n = __builtin_rint(t), z = (t - n) * 0.69314718055994530942;
    double e = 1.0 / 39916800.0;
    e = __builtin_fma(e, z, 1.0 / 3628800.0);
    e = __builtin_fma(e, z, 1.0 / 362880.0);
    e = __builtin_fma(e, z, 1.0 / 40320.0);
    e = __builtin_fma(e, z, 1.0 / 5040.0);
    e = __builtin_fma(e, z, 1.0 / 720.0);
    e = __builtin_fma(e, z, 1.0 / 120.0);
    e = __builtin_fma(e, z, 1.0 / 24.0);
    e = __builtin_fma(e, z, 1.0 / 6.0);
    e = __builtin_fma(e, z, 0.5);
    e = __builtin_fma(e, z, 1.0);
    e = __builtin_fma(e, z, 1.0);
    return __builtin_ldexp(e, (int)n);
}

// Sum over lanes 0 .. lane.
template <class T>
__device__ __forceinline__ T scan(T v, int lane) {
#pragma unroll
    for (int off = 1; off < 64; off *= 2) {
        const T up = __shfl_up(v, off);
        if (lane >= off) v += up;
    }
    return v;
}

struct Shared {
    uint32_t counts[kKeys / 2];  // two a word
    double weight[kBlocks];      // of a block's tokens, then of the blocks before it in the order
    uint32_t tokens[kBlocks];    // the same for counts
    uint16_t carried[kCarries];  // values that have kCarry more
    int carries;
    double wave_weight[kWaves];
    uint32_t wave_tokens[kWaves], wave_kept[kWaves], wave_top[kWaves];
    // Of a search: the block it ends in, the place found.
    int block, last;       // last: the last block with a weight
    double place_weight;   // of the tokens before the value
    uint32_t place_tokens; // their number
    uint32_t place_key;
    uint32_t place_count;
};

template <int DT>
struct Row {
    const uint16_t* x;
    int V, lane, wave;
    // fn(index, bits) for this wave's part of the row, 8 a lane: parts are runs in index order.
    int part, from, to;
    __device__ __forceinline__ Row(const SampleArgs& a, int row)
        : x(a.logits + row * a.ldl), V(a.V), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) {
        part = (V + kWaves * 512 - 1) / (kWaves * 512) * 512;
        from = wave * part < V ? wave * part : V;
        to = from + part < V ? from + part : V;
    }
    // Eight bits patterns at i (-infinity behind the row's end).
    __device__ __forceinline__ u32x4 load(int i) const {
        if (i + 8 <= V) return *reinterpret_cast<const u32x4_any*>(x + i);
        constexpr uint32_t low = DT == 0 ? 0xFC00u : 0xFF80u;
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = (i + 2 * e < V ? x[i + 2 * e] : low) | (i + 2 * e + 1 < V ? (uint32_t)x[i + 2 * e + 1] : low) << 16;
        return v;
    }
};

__device__ __forceinline__ uint32_t half_of(const u32x4& v, int e) { return v[e / 2] >> (16 * (e % 2)) & 0xFFFFu; }

template <int DT>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    Shared& s = *reinterpret_cast<Shared*>(raw);
    const int tid = threadIdx.x, row_at = blockIdx.x;
    const Row<DT> row(a, row_at);
    const int lane = row.lane, wave = row.wave;
    const float temperature = a.temperature ? a.temperature[row_at] : 1.0f;
    const bool greedy = !(temperature > 0.0f);

    // Count the row's values, and its largest.
    if (!greedy) {
        for (int i = tid; i < kKeys / 8; i += kThreads) reinterpret_cast<u32x4*>(s.counts)[i] = u32x4{0u, 0u, 0u, 0u};
        if (tid == 0) s.carries = 0, s.last = 0;
        __syncthreads();
    }
    uint32_t top = 0;
    for (int base = 0; base < row.part; base += 512) {  // as often for each wave
        // The one that fills a count's lower 15 bits takes them away again.
        // Between two barriers there are at most 4 * 8 * kThreads = 2^15 others,
        // so 16 bits hold them.
        if (!greedy && base % 2048 == 0 && base != 0) __syncthreads();
        const int i = row.from + base + 8 * lane;
        if (i >= row.to) continue;
        const u32x4 v = row.load(i);
        uint32_t key[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            key[e] = key_of<DT>(half_of(v, e));
            top = key[e] > top ? key[e] : top;
        }
        if (greedy) continue;
        uint32_t old[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            old[e] = key[e] != 0 ? atomicAdd(&s.counts[key[e] / 2], 1u << (16 * (key[e] & 1))) >> (16 * (key[e] & 1)) & 0xFFFFu : 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (old[e] == kCarry - 1) {
                atomicSub(&s.counts[key[e] / 2], kCarry << (16 * (key[e] & 1)));
                s.carried[atomicAdd(&s.carries, 1)] = (uint16_t)key[e];
            }
    }
#pragma unroll
    for (int off = 32; off > 0; off /= 2) {
        const uint32_t o = __shfl_xor(top, off);
        top = o > top ? o : top;
    }
    if (lane == 0) s.wave_top[wave] = top;
    __syncthreads();
    top = s.wave_top[lane % kWaves];
#pragma unroll
    for (int off = kWaves / 2; off > 0; off /= 2) {
        const uint32_t o = __shfl_xor(top, off);
        top = o > top ? o : top;
    }
    if (top == 0) {  // nothing to draw
        if (tid == 0) {
            a.tokens[row_at] = kNone;
            if (a.probs) a.probs[row_at] = 0.0f;
        }
        return;
    }

    uint32_t key = top, before = 0;  // the drawn token's value, and how many of that value come before it
    double prob = 1.0;
    if (!greedy) {
        const double most = (double)value_of<DT>(top), per = 1.4426950408889634074 / (double)temperature;
        const int carries = s.carries;
        // A value's weight and how often it occurs. Block b holds the keys
        // kKeys - 1 - 64 b - lane, so that lanes and blocks go down the order.
        auto count_at = [&](int b, int l) {
            const uint32_t k = kKeys - 1 - 64 * b - l;
            uint32_t n = s.counts[k / 2] >> (16 * (k & 1)) & 0xFFFFu;
            for (int i = 0; i < carries; ++i) n += s.carried[i] == k ? kCarry : 0u;
            return n;
        };
        auto weight_at = [&](int b, int l) {
            const uint32_t k = kKeys - 1 - 64 * b - l;
            return k == top ? 1.0 : exp2_of(((double)value_of<DT>(k) - most) * per);
        };
        const float min_p = a.min_p ? a.min_p[row_at] : 0.0f;
        const double least = min_p > 0.0f ? (min_p < 1.0f ? (double)min_p : 1.0) : 0.0;
        uint32_t kept = 0;  // tokens that min-p keeps
        for (int b = wave; b < kBlocks; b += kWaves) {
            const uint32_t n = count_at(b, lane);
            double w = 0.0;
            uint32_t sum = 0;
            if (__builtin_amdgcn_ballot_w64(n != 0) != 0) {
                const double each = n != 0 ? weight_at(b, lane) : 0.0;
                w = n * each;
                sum = n;
                kept += each >= least ? n : 0u;
#pragma unroll
                for (int off = 32; off > 0; off /= 2) {
                    w += __shfl_xor(w, off);
                    sum += __shfl_xor(sum, off);
                }
            }
            if (lane == 0) {
                s.weight[b] = w;
                s.tokens[b] = sum;
            }
        }
#pragma unroll
        for (int off = 32; off > 0; off /= 2) kept += __shfl_xor(kept, off);
        if (lane == 0) s.wave_kept[wave] = kept;
        __syncthreads();
        // Sums over the blocks before each: thread b holds block b's.
        const double own_w = s.weight[tid];
        const uint32_t own_n = s.tokens[tid];
        const double scan_w = scan(own_w, lane);
        const uint32_t scan_n = scan(own_n, lane);
        if (lane == 63) {
            s.wave_weight[wave] = scan_w;
            s.wave_tokens[wave] = scan_n;
        }
        __syncthreads();
        double to_w = 0.0;
        uint32_t to_n = 0, all_n = 0, all_kept = 0;
        for (int i = 0; i < kWaves; ++i) {
            if (i < wave) to_w += s.wave_weight[i], to_n += s.wave_tokens[i];
            all_n += s.wave_tokens[i];
            all_kept += s.wave_kept[i];
        }
        double all_w = 0.0;
        for (int i = 0; i < kWaves; ++i) all_w += s.wave_weight[i];
        const double up_w = __shfl_up(scan_w, 1);
        const uint32_t up_n = __shfl_up(scan_n, 1);
        const double from_w = lane == 0 ? to_w : to_w + up_w;
        const uint32_t from_n = lane == 0 ? to_n : to_n + up_n;
        to_w += scan_w;
        to_n += scan_n;
        s.weight[tid] = from_w;
        s.tokens[tid] = from_n;
        if (own_w > 0.0) atomicMax(&s.last, tid);

        // Finds the value with the first token at which the number of tokens
        // reaches `tokens` (by_weight false), or their weight reaches or passes
        // `weight`: place_* is then the value's, the result the value's weight.
        auto find = [&](bool by_weight, uint32_t tokens, double weight, bool pass) {
            __syncthreads();
            if (tid == 0) s.block = kBlocks;
            __syncthreads();
            const bool hit = by_weight ? (pass ? to_w > weight : to_w >= weight) : to_n >= tokens;
            if (hit && own_n != 0) atomicMin(&s.block, tid);
            __syncthreads();
            const int b = s.block < kBlocks ? s.block : s.last;  // a weight that rounding leaves above the sum of all
            const uint32_t n = count_at(b, lane);
            const double each = n != 0 ? weight_at(b, lane) : 0.0, w = n * each;
            const double in_w = scan(w, lane);
            const uint32_t in_n = scan(n, lane);
            const double before_w = s.weight[b] + (in_w - w);
            const uint32_t before_n = s.tokens[b] + (in_n - n);
            const bool here = by_weight ? (pass ? before_w + w > weight : before_w + w >= weight) : before_n + n >= tokens;
            uint64_t at = __builtin_amdgcn_ballot_w64(here && n != 0 && (!by_weight || w > 0.0));
            int l;
            if (at != 0) l = __builtin_ctzll(at);
            else l = 63 - __builtin_clzll(__builtin_amdgcn_ballot_w64(n != 0 && (!by_weight || w > 0.0)));
            if (wave == 0 && lane == l) {
                s.place_weight = before_w;
                s.place_tokens = before_n;
                s.place_key = kKeys - 1 - 64 * b - l;
                s.place_count = n;
            }
            __syncthreads();
            return __shfl(each, l);
        };
        // Weight of the first `tokens` tokens of the order.
        auto weight_of = [&](uint32_t tokens) {
            if (tokens >= all_n) return all_w;
            const double each = find(false, tokens, 0.0, false);
            return s.place_weight + (tokens - s.place_tokens) * each;
        };
        // How many tokens of the value found it takes to reach, or pass, `weight`.
        auto needed = [&](double each, double weight, bool pass) {
            const double first = s.place_weight;
            const uint32_t n = s.place_count;
            const double guess = (weight - first) / each;
            uint32_t r = guess < 1.0 ? 1u : (guess > (double)n ? n : (uint32_t)guess);
            // The quotient is off by a few at most, unless `each` is lost in the sums' rounding.
            auto there = [&](uint32_t k) { return pass ? first + k * each > weight : first + k * each >= weight; };
            for (int i = 0; i < 4 && r > 1 && there(r - 1); ++i) --r;
            for (int i = 0; i < 4 && r < n && !there(r); ++i) ++r;
            return r;
        };

        const int top_k = a.top_k ? a.top_k[row_at] : 0;
        const float top_p = a.top_p ? a.top_p[row_at] : 1.0f;
        uint32_t most_tokens = top_k > 0 && (uint32_t)top_k < all_n ? (uint32_t)top_k : all_n;
        if (top_p < 1.0f) {
            const double target = top_p > 0.0f ? (double)top_p * weight_of(most_tokens) : 0.0;
            uint32_t n = 1;
            if (target > 0.0) {
                const double each = find(true, 0u, target, false);
                n = s.place_tokens + needed(each, target, false);
            }
            most_tokens = n < most_tokens ? n : most_tokens;
        }
        if (least > 0.0 && all_kept < most_tokens) most_tokens = all_kept;
        const double total = weight_of(most_tokens);
        const float u = a.uniforms[row_at];
        const double target = (u > 0.0f ? (u < 1.0f ? (double)u : 0x0.ffffffp0) : 0.0) * total;
        const double each = find(true, 0u, target, true);
        key = s.place_key;
        before = needed(each, target, true) - 1;
        prob = each / total;
    }

    // The token: the one of its value that `before` others precede.
    uint32_t mine = 0;
    for (int i = row.from + 8 * lane; i < row.to; i += 512) {
        const u32x4 v = row.load(i);
#pragma unroll
        for (int e = 0; e < 8; ++e) mine += key_of<DT>(half_of(v, e)) == key;
    }
#pragma unroll
    for (int off = 32; off > 0; off /= 2) mine += __shfl_xor(mine, off);
    __syncthreads();  // the searches' reads of wave_tokens are done
    if (lane == 0) s.wave_tokens[wave] = mine;
    __syncthreads();
    for (int i = 0; i < wave; ++i) {
        const uint32_t n = s.wave_tokens[i];
        if (before < n) return;  // in an earlier part
        before -= n;
    }
    if (before >= mine) return;
    for (int base = row.from; base < row.to; base += 512) {
        const int i = base + 8 * lane;
        uint32_t found = 0;
        if (i < row.to) {
            const u32x4 v = row.load(i);
#pragma unroll
            for (int e = 0; e < 8; ++e) found |= (uint32_t)(key_of<DT>(half_of(v, e)) == key) << e;
        }
        const uint32_t n = __builtin_popcount(found), to = scan(n, lane), all = __shfl(to, 63);
        if (before >= all) {
            before -= all;
            continue;
        }
        if (before >= to - n && before < to) {
            for (uint32_t skip = before - (to - n); skip > 0; --skip) found &= found - 1;
            a.tokens[row_at] = i + __builtin_ctz(found);
            if (a.probs) a.probs[row_at] = (float)prob;
        }
        return;
    }
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, int dtype, hipStream_t stream) {
    hipError_t e = dtype == 0 ? allow_lds<sample_kernel<0>>(sizeof(Shared)) : allow_lds<sample_kernel<1>>(sizeof(Shared));
    if (e != hipSuccess) return e;
    if (dtype == 0) hipLaunchKernelGGL(sample_kernel<0>, dim3((unsigned)a.M), dim3(kThreads), sizeof(Shared), stream, a);
    else hipLaunchKernelGGL(sample_kernel<1>, dim3((unsigned)a.M), dim3(kThreads), sizeof(Shared), stream, a);
    return hipGetLastError();
}

}  // namespace w4a16
