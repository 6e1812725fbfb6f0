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
//
// Bound by one CU's LDS atomics and the chain of its stages (clear, count, weights,
// sums, three searches, the token's place): 64 rows of 128000 take 44.5 us, one of
// 32003 22 us, 8 to 9 where the temperature is 0 (the most probable token, without the
// histogram). A row stays on one CU: parts of it on several would exchange their
// sums of blocks of 64 values (12 KB a part) and then the counts of the blocks found.
#include "device_common.h"
#include "internal.h"

namespace w4a16 {
namespace {

typedef u32x4 u32x4_any __attribute__((aligned(2)));

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kKeys = 1 << 16;
constexpr int kBlocks = kKeys / 64;  // of 64 values each, one a thread in the scan
constexpr uint32_t kCarry = 1u << 15;
constexpr int kCarries = (int)(kSampleMaxV / kCarry) + 4;
constexpr int kNone = -1;
constexpr int kListed = 1024;  // tokens of one value that are listed

// Keys order logits as they are ordered: 0x8000 above a positive one's bits,
// a negative one's bits inverted. -infinity and what lies below it (negative
// NaN) are never drawn, nor what lies above +infinity; -0's count goes to 0's.
// The borders are multiples of 64: no block of 64 keys holds a drawn and a
// forbidden one but +infinity's, of which only the first is drawn.
template <int DT>
struct Keys {
    static constexpr uint32_t kInf = DT == 0 ? 0x7C00u : 0x7F80u;
    static constexpr uint32_t kTop = 0x8000u | kInf, kLow = 0xFFFFu - (0x8000u | kInf);  // +infinity's, -infinity's
    static constexpr uint32_t kZero = 0x8000u;
    static constexpr uint32_t kFirst = kLow + 1;
    static __device__ __forceinline__ float value(uint32_t key) {
        return act_to_float<DT>((uint16_t)(key & 0x8000u ? key & 0x7FFFu : key ^ 0xFFFFu));
    }
};
typedef short short2_t __attribute__((ext_vector_type(2)));
typedef unsigned short ushort2_t __attribute__((ext_vector_type(2)));
// The keys of two logits.
__device__ __forceinline__ uint32_t two_keys(uint32_t w) {
    return w ^ (__builtin_bit_cast(uint32_t, __builtin_bit_cast(short2_t, w) >> 15) | 0x80008000u);
}
// Where a key's count is: words of two keys; the words of block b (64 keys) are
// turned by b, so that threads that each walk through a block meet no bank twice.
__device__ __forceinline__ uint32_t word_of(uint32_t key) { return key >> 1 ^ (key >> 6 & 31u); }

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

// v of the lane that a DPP control names, 0 where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t from_lane(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double from_lane(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = from_lane<CTRL, ROWS>((uint32_t)b), hi = from_lane<CTRL, ROWS>((uint32_t)(b >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum over lanes 0 .. lane.
template <class T>
__device__ __forceinline__ T scan(T v) {
    v += from_lane<0x111, 0xF>(v);  // row_shr:1, 2, 4, 8: within 16 lanes
    v += from_lane<0x112, 0xF>(v);
    v += from_lane<0x114, 0xF>(v);
    v += from_lane<0x118, 0xF>(v);
    v += from_lane<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
    v += from_lane<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
    return v;
}
template <class T>
__device__ __forceinline__ T lane_before(T v) { return from_lane<0x138, 0xF>(v); }  // wave_shr:1
__device__ __forceinline__ double read_lane(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane), hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ uint32_t read_lane(uint32_t v, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); }

struct Shared {
    uint32_t counts[kKeys / 2];  // two a word
    double weight[kBlocks];      // of the tokens of the blocks before each in the order
    uint32_t tokens[kBlocks];    // their number
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
    int found;             // tokens of the drawn value listed
    uint32_t list[kListed];
};

template <int DT>
struct Row {
    const uint16_t* x;
    int V, lane, wave;
    // This wave's part of the row is a run of 512 logits a step, 8 a lane; as many steps for each wave.
    int steps, from;
    __device__ __forceinline__ Row(const SampleArgs& a, int row)
        : x(a.logits + row * a.ldl), V(a.V), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) {
        steps = (V + kWaves * 512 - 1) / (kWaves * 512);
        from = wave * steps * 512;
    }
    __device__ __forceinline__ int index(int step) const { return from + step * 512 + 8 * lane; }
    // Eight logits (-infinity behind the part's and the row's end).
    __device__ __forceinline__ u32x4 load(int step) const {
        const int i = step < steps ? index(step) : V;
        if (i + 8 <= V) return *reinterpret_cast<const u32x4_any*>(x + i);
        constexpr uint32_t low = 0x8000u | Keys<DT>::kInf;
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = (i + 2 * e < V ? x[i + 2 * e] : low) | (i + 2 * e + 1 < V ? (uint32_t)x[i + 2 * e + 1] : low) << 16;
        return v;
    }
    // Of N steps; a branch for all of them, so that the loads are in flight together.
    template <int N>
    __device__ __forceinline__ void load(int step, u32x4 (&v)[N]) const {
        if (step + N <= steps && from + (step + N) * 512 <= V) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = *reinterpret_cast<const u32x4_any*>(x + index(step + i));
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = load(step + i);
        }
    }
};
constexpr int kAtOnce = 4;  // steps whose loads are in flight together

template <int DT>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
    using K = Keys<DT>;
    extern __shared__ __align__(16) unsigned char raw[];
    Shared& s = *reinterpret_cast<Shared*>(raw);
    const int tid = threadIdx.x, row_at = blockIdx.x;
    const Row<DT> row(a, row_at);
    const int lane = row.lane, wave = row.wave;
    const float temperature = a.temperature ? a.temperature[row_at] : 1.0f;
    const bool greedy = !(temperature > 0.0f);
    // A key that may be drawn.
    auto drawn = [](uint32_t key) { return key - K::kFirst <= K::kTop - K::kFirst; };

    uint32_t top = 0;  // the largest logit's key
    if (greedy) {
        // The least distance below +infinity's key, two logits at once: forbidden
        // tokens' are larger than any that may be drawn.
        ushort2_t least{0xFFFF, 0xFFFF};
        for (int step = 0; step < row.steps; step += 2 * kAtOnce) {
            u32x4 v[2 * kAtOnce];
            row.load(step, v);
#pragma unroll
            for (int i = 0; i < 2 * kAtOnce; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    least = __builtin_elementwise_min(least, ushort2_t{K::kTop, K::kTop} - __builtin_bit_cast(ushort2_t, two_keys(v[i][e])));
        }
        uint32_t down = least[0] < least[1] ? least[0] : least[1];
#pragma unroll
        for (int off = 32; off > 0; off /= 2) {
            const uint32_t o = __shfl_xor(down, off);
            down = o < down ? o : down;
        }
        if (lane == 0) s.wave_top[wave] = down;
        if (tid == 0) s.found = 0;
        __syncthreads();
        for (int i = 0; i < kWaves; ++i) down = s.wave_top[i] < down ? s.wave_top[i] : down;
        top = down <= K::kTop - K::kFirst ? K::kTop - down : 0u;
        if (top == K::kZero - 1) top = K::kZero;
    } else {
        u32x4 next[kAtOnce];  // the next steps' logits are on their way while these are counted
        row.load(0, next);
        for (int i = tid; i < kKeys / 8; i += kThreads) reinterpret_cast<u32x4*>(s.counts)[i] = u32x4{0u, 0u, 0u, 0u};
        if (tid == 0) s.carries = 0, s.last = 0, s.found = 0, s.block = kBlocks;
        __syncthreads();
        // Count the row's values.
        for (int step = 0; step < row.steps; step += kAtOnce) {  // as often for each wave
            u32x4 v[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) v[i] = next[i];
            row.load(step + kAtOnce, next);
            if (step != 0) {
                // 2^15 logits raise a count by as much at most: taken out of the
                // counts that have reached it, the next ones fit too.
                static_assert(kAtOnce * 8 * kThreads <= (int)kCarry, "counts of 16 bits");
                __syncthreads();
                for (int i = 0; i < 32; ++i) {
                    const uint32_t word = 32 * tid + (i ^ (tid & 31)), n = s.counts[word];
                    if ((n & 0x80008000u) == 0) continue;
                    const uint32_t k = 2 * (32 * tid + i);
                    s.counts[word] = n & 0x7FFF7FFFu;
                    if (n & 0x8000u) s.carried[atomicAdd(&s.carries, 1)] = (uint16_t)k;
                    if (n >> 31) s.carried[atomicAdd(&s.carries, 1)] = (uint16_t)(k + 1 == K::kZero - 1 ? K::kZero : k + 1);
                }
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t k = two_keys(v[i][e]), lo = k & 0xFFFFu, hi = k >> 16;
                    // Forbidden tokens may be most of a row: they are not counted.
                    if (lo != K::kLow) atomicAdd(&s.counts[word_of(lo)], lo & 1 ? 0x10000u : 1u);
                    if (hi != K::kLow) atomicAdd(&s.counts[word_of(hi)], hi & 1 ? 0x10000u : 1u);
                }
        }
        __syncthreads();
        if (tid == 0) {  // both zeros are one value; each may have 2^15 - 1, and 2^15 of the last steps
            const uint32_t at = word_of(K::kZero), from = word_of(K::kZero - 1);
            uint32_t both = (s.counts[from] >> 16) + (s.counts[at] & 0xFFFFu);
            for (; both > 0xFFFFu; both -= kCarry) s.carried[s.carries++] = (uint16_t)K::kZero;
            s.counts[from] &= 0xFFFFu;
            s.counts[at] = (s.counts[at] & 0xFFFF0000u) | both;
        }
        __syncthreads();
    }

    uint32_t key = top, before = 0, same = ~0u;  // the drawn token's value, how many of that value come before it, how many there are
    double prob = 1.0;
    if (!greedy) {
        // Block b holds the keys kKeys - 1 - 64 b - i, i = 0 .. 63, so that blocks
        // and i go down the order. Thread b holds block b's counts.
        const int carries = s.carries;
        if (carries > 0) {  // NaNs among them, which lie in +infinity's block too: 0 is no value that may be drawn
            for (int i = tid; i < carries; i += kThreads)
                if (!drawn(s.carried[i])) s.carried[i] = 0;
            __syncthreads();
        }
        auto carried = [&](uint32_t k) {
            uint32_t n = 0;
            for (int i = 0; i < carries; ++i) n += s.carried[i] == k ? kCarry : 0u;
            return n;
        };
        const uint32_t high = kKeys - 1 - 64 * tid;  // the block's first key
        uint32_t counts[32];                         // of the keys high - 2 i (upper half) and high - 2 i - 1
        uint32_t any = 0;
        const bool forbidden = !drawn(high - 63);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            counts[i] = forbidden ? 0u : s.counts[word_of(high - 2 * i)];
            if (high - 63 == K::kTop) counts[i] = i == 31 ? counts[i] & 0xFFFFu : 0u;  // behind +infinity
            any |= counts[i];
        }
        if (carries > 0 && !forbidden)
            for (int i = 0; i < carries; ++i) any |= (high - s.carried[i]) < 64u;
        if (any != 0) atomicMin(&s.block, tid);
        __syncthreads();
        const int first_block = s.block;
        if (first_block == kBlocks) {  // nothing to draw
            if (tid == 0) {
                a.tokens[row_at] = kNone;
                if (a.probs) a.probs[row_at] = 0.0f;
            }
            return;
        }
        if (tid == first_block) {
            uint32_t k = 0;
#pragma unroll
            for (int i = 31; i >= 0; --i) {
                if (counts[i] & 0xFFFFu) k = high - 2 * i - 1;
                if (counts[i] >> 16) k = high - 2 * i;
            }
            for (int i = 0; i < carries; ++i)
                if (high - s.carried[i] < 64u && s.carried[i] > k) k = s.carried[i];
            s.place_key = k;
        }
        __syncthreads();
        top = s.place_key;
        // A value's weight. Within a block the values are equally far apart, so
        // its weights are a power series: two exponentials a block.
        const double most = (double)K::value(top), per = 1.4426950408889634074 / (double)temperature;
        auto weight_at = [&](uint32_t k) { return k == top ? 1.0 : exp2_of(((double)K::value(k) - most) * per); };
        const float min_p = a.min_p ? a.min_p[row_at] : 0.0f;
        const double least = min_p > 0.0f ? (min_p < 1.0f ? (double)min_p : 1.0) : 0.0;
        double own_w = 0.0;
        uint32_t own_n = 0, kept = 0;  // kept: tokens that min-p keeps
        if (any != 0) {
            const double ratio = exp2_of(((double)K::value(high - 63) - (double)K::value(high - 62)) * per);
            const bool lists = carries > 0, sieve = least > 0.0;
            // From the block's first key on, or the row's largest logit's.
            const int skip = high > top ? (int)(high - top) : 0;
            double w = weight_at(high - skip);
#pragma unroll
            for (int i = 0; i < 64; ++i) {
                if (i % 8 == 0) __builtin_amdgcn_sched_barrier(0);  // 128 registers a thread: no more at once
                uint32_t n = i % 2 == 0 ? counts[i / 2] >> 16 : counts[i / 2] & 0xFFFFu;
                if (lists) n += carried(high - i);
                own_n += n;
                own_w = __builtin_fma((double)n, w, own_w);
                if (sieve) kept += w >= least ? n : 0u;
                w = i < skip ? w : w * ratio;
            }
        }
        // Sums over the blocks before each.
        const double scan_w = scan(own_w);
        const uint32_t scan_n = scan(own_n), scan_kept = scan(kept);
        if (lane == 63) {
            s.wave_weight[wave] = scan_w;
            s.wave_tokens[wave] = scan_n;
            s.wave_kept[wave] = scan_kept;
        }
        if (own_w > 0.0) atomicMax(&s.last, tid);
        __syncthreads();
        double to_w = 0.0, all_w = 0.0;
        uint32_t to_n = 0, all_n = 0, all_kept = 0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            if (i == wave) to_w = all_w, to_n = all_n;
            all_w += s.wave_weight[i];
            all_n += s.wave_tokens[i];
            all_kept += s.wave_kept[i];
        }
        const double from_w = to_w + lane_before(scan_w);  // lane 0: nothing
        const uint32_t from_n = to_n + lane_before(scan_n);
        to_w += scan_w;
        to_n += scan_n;
        s.weight[tid] = from_w;
        s.tokens[tid] = from_n;

        // Finds the value with the first token at which the number of tokens
        // reaches `tokens` (by_weight false), or their weight reaches or passes
        // `weight`: place_* is then the value's, the result the value's weight.
        auto find = [&](bool by_weight, uint32_t tokens, double weight, bool pass) {
            __syncthreads();
            if (tid == 0) s.block = kBlocks;
            __syncthreads();
            const bool hit = by_weight ? (pass ? to_w > weight : to_w >= weight) : to_n >= tokens;
            const uint64_t hits = __builtin_amdgcn_ballot_w64(hit && own_n != 0);
            if (hits != 0 && lane == 0) atomicMin(&s.block, 64 * wave + __builtin_ctzll(hits));
            __syncthreads();
            const int b = s.block < kBlocks ? s.block : s.last;  // a weight that rounding leaves above the sum of all
            const uint32_t k = kKeys - 1 - 64 * b - lane;
            uint32_t n = s.counts[word_of(k)] >> (16 * (k & 1)) & 0xFFFFu;
            if (kKeys - 64 - 64 * b == (int)K::kTop && lane != 63) n = 0;  // behind +infinity
            if (carries > 0) n += carried(k);
            const double each = n != 0 ? weight_at(k) : 0.0, w = n * each;
            const double in_w = scan(w);
            const uint32_t in_n = scan(n);
            const double before_w = s.weight[b] + lane_before(in_w);
            const uint32_t before_n = s.tokens[b] + lane_before(in_n);
            const bool here = by_weight ? (pass ? before_w + w > weight : before_w + w >= weight) : before_n + n >= tokens;
            const bool some = n != 0 && (!by_weight || w > 0.0);
            const uint64_t at = __builtin_amdgcn_ballot_w64(here && some);
            const int l = at != 0 ? __builtin_ctzll(at) : 63 - __builtin_clzll(__builtin_amdgcn_ballot_w64(some) | 1);
            if (wave == 0 && lane == l) {
                s.place_weight = before_w;
                s.place_tokens = before_n;
                s.place_key = k;
                s.place_count = n;
            }
            __syncthreads();
            return read_lane(each, l);
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
        double total = weight_of(most_tokens);
        if (top_p < 1.0f) {
            const double target = top_p > 0.0f ? (double)top_p * total : 0.0;
            uint32_t n = 1;
            if (target > 0.0) {
                const double each = find(true, 0u, target, false);
                const uint32_t r = needed(each, target, false);
                n = s.place_tokens + r;
                if (n < most_tokens) total = s.place_weight + r * each;
            } else {
                total = 1.0;
            }
            most_tokens = n < most_tokens ? n : most_tokens;
        }
        if (least > 0.0 && all_kept < most_tokens) {
            most_tokens = all_kept;
            total = weight_of(most_tokens);
        }
        const float u = a.uniforms[row_at];
        const double target = (u > 0.0f ? (u < 1.0f ? (double)u : 0x0.ffffffp0) : 0.0) * total;
        const double each = find(true, 0u, target, true);
        key = s.place_key;
        same = s.place_count;
        before = needed(each, target, true) - 1;
        prob = each / total;
    } else if (top == 0) {
        if (tid == 0) {
            a.tokens[row_at] = kNone;
            if (a.probs) a.probs[row_at] = 0.0f;
        }
        return;
    }

    // The token: the one of its value that `before` others precede.
    const uint32_t bits = key & 0x8000u ? key & 0x7FFFu : key ^ 0xFFFFu, two = bits | bits << 16;
    const uint32_t sign = key == K::kZero ? 0x7FFF7FFFu : ~0u;  // a zero of either sign
    auto matches = [&](const u32x4& v) {  // which of the eight
        uint32_t m = 0;
        bool some = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t x = (v[e] & sign) ^ two;
            some |= (x & 0xFFFFu) == 0 || x < 0x10000u;
        }
        if (some) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t x = (v[e] & sign) ^ two;
                m |= (uint32_t)((x & 0xFFFFu) == 0) << (2 * e) | (uint32_t)(x < 0x10000u) << (2 * e + 1);
            }
        }
        return m;
    };
    auto answer = [&](int index) {
        a.tokens[row_at] = index;
        if (a.probs) a.probs[row_at] = (float)prob;
    };
    // Few of that value: list them, and take the one with `before` smaller ones.
    const bool listed = same <= kListed;
    uint32_t mine = 0;
    for (int step = 0; step < row.steps; step += 2 * kAtOnce) {
        u32x4 v[2 * kAtOnce];
        row.load(step, v);
#pragma unroll
        for (int i = 0; i < 2 * kAtOnce; ++i) {
            uint32_t m = step + i < row.steps ? matches(v[i]) : 0u;
            mine += __builtin_popcount(m);
            for (; listed && m != 0; m &= m - 1) s.list[atomicAdd(&s.found, 1)] = row.index(step + i) + __builtin_ctz(m);
        }
    }
    if (listed) {
        __syncthreads();
        const int n = s.found;
        for (int i = tid; i < n; i += kThreads) {
            const uint32_t index = s.list[i];
            uint32_t smaller = 0;
            for (int j = 0; j < n; ++j) smaller += s.list[j] < index;
            if (smaller == before) answer((int)index);
        }
        return;
    }
    // Many: the wave's part that holds it, then the step.
    mine = read_lane(scan(mine), 63);
    __syncthreads();  // the searches' reads of wave_tokens are done
    if (lane == 0) s.wave_tokens[wave] = mine;
    __syncthreads();
    for (int i = 0; i < wave; ++i) {
        const uint32_t n = s.wave_tokens[i];
        if (before < n) return;  // in an earlier part
        before -= n;
    }
    if (before >= mine) return;
    for (int step = 0; step < row.steps; ++step) {
        uint32_t m = matches(row.load(step));
        const uint32_t n = __builtin_popcount(m), to = scan(n), all = read_lane(to, 63);
        if (before >= all) {
            before -= all;
            continue;
        }
        if (before >= to - n && before < to) {
            for (uint32_t skip = before - (to - n); skip > 0; --skip) m &= m - 1;
            answer(row.index(step) + __builtin_ctz(m));
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
