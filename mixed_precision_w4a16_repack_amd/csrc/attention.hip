// attention.hip -- attention of one new token per sequence over the paged
// key/value cache (layout in include/w4a16.h, kv_layout.h):
//   s_t = scale * q . k_t,  o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),
// over the tokens t a sequence sees, in one pass with a running reference m.
//
// Tiles of 32 tokens. A cache tile is an MFMA operand as it is stored, so
// nothing is shuffled: S^T = K Q^T (16 tokens x 16 query heads of one kv
// head), whose result already lies as the B operand of O^T += V^T P^T (the
// value tiles hold their tokens in that order). Keys, values and results stay
// in registers; a wave loads a tile's keys while it works on the one before.
//
// Scores are in base 2 (scale * log2(e) folded into one factor). The running
// reference moves only when a score passes it by kHeadroom, which is rare
// after the first tiles, so a tile usually costs no cross-lane step and no
// rescaling of O. 16-bit probabilities carry a factor 2^13 in fp16, which
// keeps them out of the subnormals down to 2^-27 of the largest (and not lost
// above 2^-38); the sums take the unrounded fp32 ones.
//
// A probability is two operands, a 16-bit number and the rest's, and the
// product with the values is made with both: one alone moves the result by as
// much as the result's own rounding does. The matrix cores have the time (64 x
// 2048 tokens, 16 bits: 80.9 us with one, 81.2 with two; int8, D = 64: 25.5 and
// 26.2; 333 tokens of one sequence 7.1 and 7.35). Over int8 with bf16 results
// it is one fp16 operand: its 2^-11 is an eighth of the result's half step, and
// the second one would cost 1.5 % (with two head tiles 4.5 %).
//
// int8: codes become exact fp16 values (0x6400 | (code ^ 0x80) is 1152 + code),
// the key's scale multiplies the score, and the value's scale its probability,
// w = p * vs. Scales of any size must not leave fp16's range, so w has a
// reference of its own, c >= log2(w): w is formed as p * vs * f with
// f = 2^(13 - c + m). A bf16 query is moved by a power of two to the top of
// fp16's range (its 8 bits are exact there; elements below 2^-29 of the
// largest lose bits).
//
// What bounds it: the cache's bytes. 64 sequences of 2048 tokens, 8 kv heads
// of 128: 81 us in 16 bits (6.6 TB/s; a plain read of as much reaches 6.9),
// 44 us in int8 (6.3 TB/s). The loads are non-temporal (each byte is read
// once; through the caches as usual they take 10 us more).
//
// Work is divided by tiles over a fixed number of workgroups, computed on the
// device from the lengths (the host does not know them): each takes an equal
// run of the list of all (sequence, kv head, tile), whatever the lengths are,
// or, where there are few heads or few tiles, an equal part of one head.
// A head's start (query, page table, first tile: three waits) and end (four
// waves joined) count as kHeadBytes more: without that, 64 sequences from 0 to
// 6000 tokens took 112 us, the workgroups of the short ones being last, and
// now take 91 (80 us at 6.5 TB/s). A (sequence, head) that several workgroups
// share is joined by the last of them to arrive, in order of position, so the
// result does not depend on the order of arrival: kFan at a time, over levels,
// each level about 3 us (one sequence of 131000 tokens, int8: 52 us, of them 6
// in two levels; with 16 at a time 55, with 64 in one level 63).
// A short call is bound by its chain of waits: 333 tokens of one sequence
// 7.35 us, of them 2 before the first instruction and after the last, 1.3 to
// find its share, 2.9 for three tiles a wave and 1 to join the waves.
#include "device_common.h"
#include "exchange.h"
#include "internal.h"
#include "kv_layout.h"

namespace w4a16 {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;              // tokens
// Least tiles per workgroup when a head is split: a split costs a join. With 8,
// 333 tokens took 0.9 us more (of 7.1); with 32, 1000 tokens 11.5 and not 9.6.
constexpr int kMinTiles = 16;
constexpr int kHeadBytes = 80 << 10;   // a head's start and end cost a workgroup about as much as reading this
constexpr int kFan = 8;                // partial results joined at once (their loads are in flight together)
constexpr int kChunkBits = 24;         // a sum over sequences: slots << kChunkBits | chunks, the latter cut to kChunkMost a lane
constexpr int64_t kChunkMask = ((int64_t)1 << kChunkBits) - 1, kChunkMost = 1 << 16;
constexpr float kLowest = -3.402823466e38f;

typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

// How many workgroups of each kernel share a CU. More waves than the bytes in
// flight need make the reads slower, not faster: int8 D = 128 takes 63 us with
// three and 46 with two at 64 x 2048 tokens (49 with one), int8 D = 64 60 us
// with four, 52 with three, 47 with two. The larger operands' registers allow
// one; 16 bits with two head tiles lose by a second one too (64 x 4096 tokens
// of one kv head, 32 query heads: 37 and 39 us), int8 gains (34 and 28 us).
template <int KIND, int D, int HT>
constexpr int kPerCU = D > 192 || (D > 128 && (HT == 2 || KIND == 0)) || (HT == 2 && KIND == 0) ? 1 : 2;

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

// What a sequence of a length sees: tokens lo .. n - 1, in the tiles
// [first, first + count).
struct Span {
    int n, lo, first, count;
    __device__ __forceinline__ Span(const AttentionArgs& a, int length) {
        n = length < 0 ? 0 : (length > a.most ? a.most : length);
        lo = n > a.reach ? n - a.reach : 0;
        first = lo / kTile;
        count = n > lo ? (n - 1) / kTile + 1 - first : 0;
    }
};

// Two probabilities as NP packed operands, each what the ones before leave.
// fp16 is cut, not rounded (one instruction a pair): the next operand takes
// what is cut off.
template <int PDT, int NP>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&out)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        if constexpr (PDT == 0 && NP > 1) {
            const auto h = __builtin_amdgcn_cvt_pkrtz(x, y);
            out[i] = __builtin_bit_cast(uint32_t, h);
            x = __builtin_fmaf((float)h[0], -1.0f, x);
            y = __builtin_fmaf((float)h[1], -1.0f, y);
        } else {
            const uint16_t a = to_act_bits<PDT>(x), b = to_act_bits<PDT>(y);
            out[i] = (uint32_t)a | (uint32_t)b << 16;
            x -= act_to_float<PDT>(a);
            y -= act_to_float<PDT>(b);
        }
    }
}

// What a head of n tiles counts for in the two ways to divide the work.
__device__ __forceinline__ int chunks_of(int n) { return (n + kMinTiles - 1) / kMinTiles; }

template <int DT, int KIND, int D, int HT>
struct Attend {
    static constexpr int kHeadCost = kHeadBytes / (kTile * D * (KIND == 1 ? 2 : 4));  // in tiles
    static __device__ __forceinline__ int slots_of(int n) { return n > 0 ? n + kHeadCost : 0; }
    static constexpr bool kI8 = KIND == 1;
    static constexpr bool kF16P = kI8 || DT == 0;
    static constexpr int PDT = kF16P ? 0 : 1;             // operand type of both products
    static constexpr int NP = kI8 && DT == 1 ? 1 : 2;     // operands of a probability
    static constexpr int NL = D * (kI8 ? 1 : 2) / 32;     // 16-byte loads a lane for a tile's keys (and its values)
    static constexpr int NQ = D / 32;                     // MFMAs along d
    static constexpr int NO = D / 16;
    static constexpr int kCols = 16 * HT;
    static constexpr int kLd = D + 4;                     // floats between heads in LDS: spreads them over the banks
    using L = KvPlace<KIND>;
    using Pr = Prob<kF16P>;

    const AttentionArgs& a;
    const int lane, wave, g, col;
    u32x4 q[HT][NQ];
    float factor[HT];
    u32x4 kb[NL], vb[NL];
    floatx4 ks[2], vs[2];
    floatx4 o[HT][NO];
    float m[HT], l[HT], c[HT], f[HT];

    __device__ __forceinline__ explicit Attend(const AttentionArgs& args)
        : a(args), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), g(lane >> 4), col(lane & 15) {}

    // The queries of sequence b, heads head0 .. head0 + heads - 1 (heads <= kCols) as B operands.
    __device__ __forceinline__ void load_query(int64_t b, int head0, int heads) {
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            const bool in = 16 * h + col < heads;
            const uint16_t* p = a.q + b * a.q_ts + (int64_t)(head0 + 16 * h + col) * a.q_hs + 8 * g;
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                q[h][i] = u32x4{0u, 0u, 0u, 0u};
                if (in) q[h][i] = *reinterpret_cast<const u32x4_any*>(p + 32 * i);
            }
            m[h] = kLowest;
            c[h] = kLowest;
            l[h] = 0.0f;
            f[h] = 1.0f;
#pragma unroll
            for (int i = 0; i < NO; ++i) o[h][i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }

    __device__ __forceinline__ void convert_query() {
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            factor[h] = a.scale * 1.44269504088896341f;
            if constexpr (kI8 && DT == 1) {
                uint32_t top = 0u;
#pragma unroll
                for (int i = 0; i < NQ; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t x = q[h][i][e] & 0x7FFFu, y = q[h][i][e] >> 16 & 0x7FFFu;
                        top = x > top ? x : top;
                        top = y > top ? y : top;
                    }
                uint32_t t = __shfl_xor(top, 16);
                top = t > top ? t : top;
                t = __shfl_xor(top, 32);
                top = t > top ? t : top;
                const int e = (int)(top >> 7);  // biased exponent of the head's largest element
                const int up = e == 255 || top == 0u ? 0 : 14 + 127 - e;
#pragma unroll
                for (int i = 0; i < NQ; ++i)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t bits = q[h][i][w];
                        const float x = __builtin_ldexpf(__builtin_bit_cast(float, bits << 16), up);
                        const float y = __builtin_ldexpf(__builtin_bit_cast(float, bits & 0xFFFF0000u), up);
                        q[h][i][w] = (uint32_t)to_act_bits<0>(x) | (uint32_t)to_act_bits<0>(y) << 16;
                    }
                factor[h] = __builtin_ldexpf(factor[h], -up);
            }
        }
    }

    __device__ __forceinline__ void load_keys(const unsigned char* rec, int sub, int unit) {
        const u32x4* p = reinterpret_cast<const u32x4*>(rec + (int64_t)sub * NL * 1024) + unit;
#pragma unroll
        for (int i = 0; i < NL; ++i) kb[i] = __builtin_nontemporal_load(p + 64 * i);
    }
    __device__ __forceinline__ void load_values(const unsigned char* rec, int sub, int unit) {
        if constexpr (kI8) {  // first: they are needed first

            const float* sc = reinterpret_cast<const float*>(rec + 2 * L::keys_bytes(D, a.P)) + sub * kTile + 4 * g;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ks[i] = *reinterpret_cast<const floatx4*>(sc + 16 * i);
                vs[i] = *reinterpret_cast<const floatx4*>(sc + a.P + 16 * i);
            }
        }
        const u32x4* p = reinterpret_cast<const u32x4*>(rec + L::keys_bytes(D, a.P) + (int64_t)sub * NL * 1024) + unit;
#pragma unroll
        for (int i = 0; i < NL; ++i) vb[i] = __builtin_nontemporal_load(p + 64 * i);
    }

    // s[h][0..3]: tokens 4g .. 4g+3 of the tile, s[h][4..7]: 16 tokens on.
    __device__ __forceinline__ void scores(float (&s)[HT][8]) {
        floatx4 acc[HT][2];
#pragma unroll
        for (int h = 0; h < HT; ++h)
#pragma unroll
            for (int t = 0; t < 2; ++t) acc[h][t] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                u32x4 k;
                if constexpr (kI8) {
                    const u32x4& w = kb[t * (NQ / 2) + i / 2];
                    k = i % 2 == 0 ? codes8_to_f16(w[0], w[1]) : codes8_to_f16(w[2], w[3]);
                } else {
                    k = kb[t * NQ + i];
                }
#pragma unroll
                for (int h = 0; h < HT; ++h) acc[h][t] = mfma16x16x32<PDT>(k, q[h][i], acc[h][t]);
            }
#pragma unroll
        for (int h = 0; h < HT; ++h)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[h][j] = acc[h][j / 4][j % 4];
    }

    // Scores to base 2, then to the probabilities' operands; `partial` tiles
    // see only tokens from lo to hi - 1 of the tile.
    __device__ __forceinline__ void probabilities(float (&s)[HT][8], u32x4 (&p)[HT][NP], bool partial, int lo, int hi) {
        uint32_t seen = 0xFFu;
        if (partial) {
            seen = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int t = j / 4 * 16 + 4 * g + j % 4;
                seen |= (uint32_t)(t >= lo && t < hi) << j;
            }
            if constexpr (kI8) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (!(seen >> j & 1u)) vs[j / 4][j % 4] = 0.0f;
            } else {
                // An unseen value may be anything, and 0 * NaN is NaN.
                uint32_t keep[4];
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    keep[w] = (seen >> (2 * w) & 1u ? 0xFFFFu : 0u) | (seen >> (2 * w + 1) & 1u ? 0xFFFF0000u : 0u);
#pragma unroll
                for (int i = 0; i < NL; ++i)
#pragma unroll
                    for (int w = 0; w < 4; ++w) vb[i][w] &= keep[w];
            }
        }
        float peak[HT];
        bool above = false;
#pragma unroll
        for (int h = 0; h < HT; ++h) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (kI8) s[h][j] *= ks[j / 4][j % 4] * factor[h];
                else s[h][j] *= factor[h];
            }
            if (partial) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (!(seen >> j & 1u)) s[h][j] = -INFINITY;
            }
            peak[h] = s[h][0];
#pragma unroll
            for (int j = 1; j < 8; ++j) peak[h] = fmaxf(peak[h], s[h][j]);
            above |= peak[h] > m[h] + Pr::kHeadroom;
        }
        float e[HT][8], w[HT][8];
        auto weigh = [&]() {
#pragma unroll
            for (int h = 0; h < HT; ++h) {
                const float ref = kI8 ? m[h] : m[h] - Pr::kBias;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    e[h][j] = exp2_fast(s[h][j] - ref);
                    w[h][j] = kI8 ? e[h][j] * vs[j / 4][j % 4] * f[h] : e[h][j];
                }
            }
        };
        if constexpr (kI8) {
            weigh();
#pragma unroll
            for (int h = 0; h < HT; ++h) {
                float top = w[h][0];
#pragma unroll
                for (int j = 1; j < 8; ++j) top = fmaxf(top, w[h][j]);
                above |= top > 0x1p15f;
            }
        }
        if (__builtin_amdgcn_ballot_w64(above) != 0) {  // move the references: rare after the first tiles
#pragma unroll
            for (int h = 0; h < HT; ++h) {
                const float mn = column_max(fmaxf(m[h], peak[h]));
                const float keep_l = exp2_fast(m[h] - mn);
                float keep_o = keep_l;
                if constexpr (kI8) {
                    float y = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) y = fmaxf(y, exp2_fast(s[h][j] - mn) * vs[j / 4][j % 4]);
                    // f stays within fp32: c is at least mn - 113
                    const float cn = fmaxf(fmaxf(c[h], mn + __builtin_amdgcn_logf(column_max(y))), mn - 113.0f);
                    keep_o = exp2_fast(c[h] - cn);
                    c[h] = cn;
                    f[h] = exp2_fast(Pr::kBias - (cn - mn));
                }
                m[h] = mn;
                l[h] *= keep_l;
#pragma unroll
                for (int i = 0; i < NO; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[h][i][r] *= keep_o;
            }
            if constexpr (kI8) weigh();
        }
        if constexpr (!kI8) weigh();
#pragma unroll
        for (int h = 0; h < HT; ++h) {
#pragma unroll
            for (int j = 0; j < 8; ++j) l[h] += e[h][j];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t parts[NP];
                split_pair<PDT, NP>(w[h][2 * x], w[h][2 * x + 1], parts);
#pragma unroll
                for (int i = 0; i < NP; ++i) p[h][i][x] = parts[i];
            }
        }
    }

    __device__ __forceinline__ void accumulate(const u32x4 (&p)[HT][NP]) {
        // A product should not wait for the one before it: with one head tile
        // the second operands' products come after all of the first ones'
        // (64 ragged sequences: 90 us side by side, 87.6 so); with two they
        // take turns, and the other order spills at D = 256 (30 and 40 us).
        constexpr int kPasses = HT == 1 ? NP : 1, kEach = NP / kPasses;
#pragma unroll
        for (int pass = 0; pass < kPasses; ++pass)
#pragma unroll
            for (int i = 0; i < NO; ++i) {
                u32x4 v;
                if constexpr (kI8) {
                    const u32x4& w = vb[i / 2];
                    v = i % 2 == 0 ? codes8_to_f16(w[0], w[1]) : codes8_to_f16(w[2], w[3]);
                } else {
                    v = vb[i];
                }
#pragma unroll
                for (int j = 0; j < kEach; ++j)
#pragma unroll
                    for (int h = 0; h < HT; ++h) o[h][i] = mfma16x16x32<PDT>(v, p[h][pass * kEach + j], o[h][i]);
            }
    }

    // This wave's share of tiles [from, to) of sequence b: every kWaves-th,
    // those of missing pages left out.
    __device__ __forceinline__ void run(int64_t b, int kv_head, const Span& sp, int from, int to) {
        const int tiles_per_page = a.P / kTile;
        const int whole_shift = (tiles_per_page & (tiles_per_page - 1)) == 0 ? __builtin_ctz(tiles_per_page) : -1;
        int block = from + wave;  // first tile of the 64 in hand, lane i holding block + kWaves * i
        uint64_t todo = 0;
        int64_t place = 0;
        int sub_l = 0;
        auto fetch = [&]() {
            while (todo == 0 && block < to) {
                const int tile = block + kWaves * lane;
                int64_t page = -1;
                if (tile < to) {
                    const int at = whole_shift >= 0 ? tile >> whole_shift : tile / tiles_per_page;
                    page = a.table[b * a.table_ld + at];
                    sub_l = tile - at * tiles_per_page;
                }
                const bool ok = page >= 0 && page < a.pages;
                place = ok ? (page * a.H + kv_head) * L::record_bytes(D, a.P) : 0;
                todo = __builtin_amdgcn_ballot_w64(ok);
                if (todo == 0) block += 64 * kWaves;
            }
        };
        const unsigned char* rec = nullptr;
        int sub = 0, tile = 0;
        auto next = [&]() -> bool {  // the next tile's place, if there is one
            if (todo == 0) fetch();
            if (todo == 0) return false;
            const int i = __builtin_ctzll(todo);
            todo &= todo - 1;
            rec = a.cache + read_lane(place, i);
            sub = __builtin_amdgcn_readlane(sub_l, i);
            tile = block + kWaves * i;
            if (todo == 0) block += 64 * kWaves;
            return true;
        };
        if (!next()) return;
        load_keys(rec, sub, lane);
        issue_fence();
        load_values(rec, sub, lane);
        issue_fence();
        convert_query();
        bool more = true;
        do {
            const int at = tile * kTile;
            float s[HT][8];
            u32x4 p[HT][NP];
            // After the last tile every lane loads that tile's first unit
            // again (one cache line): loads on a condition would have to be
            // waited for as if they were the newest.
            more = next();
            const int unit = more ? lane : 0;
            scores(s);
            issue_fence();
            load_keys(rec, sub, unit);
            issue_fence();
            const int lo = sp.lo - at, hi = sp.n - at;
            probabilities(s, p, lo > 0 || hi < kTile, lo, hi);
            accumulate(p);
            issue_fence();
            load_values(rec, sub, unit);
            issue_fence();
        } while (more);
    }

    // The four waves' results in LDS, relative to each wave's reference.
    __device__ __forceinline__ void to_lds(float* lds, int heads) {
        float* ml = lds + kWaves * heads * kLd;
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            l[h] = column_sum(l[h]);
            const int head = 16 * h + col;
            if (head < heads) {
                const float back = kI8 ? exp2_fast(c[h] - Pr::kBias - m[h]) : 1.0f;
                float* p = lds + (wave * heads + head) * kLd + 4 * g;
#pragma unroll
                for (int i = 0; i < NO; ++i) {
                    floatx4 v = o[h][i];
                    if constexpr (kI8) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] *= back;
                    }
                    *reinterpret_cast<floatx4*>(p + 16 * i) = v;
                }
                if (g == 0) {
                    ml[2 * (wave * heads + head)] = m[h];
                    ml[2 * (wave * heads + head) + 1] = l[h];
                }
            }
        }
    }
};

// A running join of partial results (m, l, o): sums relative to m.
struct Join {
    float m = kLowest, l = 0.0f;
    floatx4 o{0.0f, 0.0f, 0.0f, 0.0f};
    __device__ __forceinline__ void add(float pm, float pl, const floatx4& po) {
        const float w = exp2_fast(pm - m);
        l += w * pl;
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] += w * po[r];
    }
};

template <int DT>
__device__ __forceinline__ void store_out(const AttentionArgs& a, int64_t b, int head, int d, const Join& j) {
    const float inv = 1.0f / (j.l == 0.0f ? 1.0f : j.l);
    u32x2 v;
#pragma unroll
    for (int x = 0; x < 2; ++x)
        v[x] = (uint32_t)to_act_bits<DT>(j.o[2 * x] * inv) | (uint32_t)to_act_bits<DT>(j.o[2 * x + 1] * inv) << 16;
    *reinterpret_cast<u32x2_any*>(a.out + b * a.o_ts + (int64_t)head * a.o_hs + d) = v;
}

// Workspace: counters (two per workgroup and level), then two partial results
// per workgroup (0: of a head begun by an earlier workgroup, 1: of one that
// begins here): per head two pairs (m, l), for even and odd levels of the join
// (other waves may still read the one while the next is written), then D floats.
template <int D, int HT>
struct Partial {
    static constexpr int kStride = D + 4;
    static constexpr int64_t kFloats = 16 * HT * kStride;
    static __device__ __forceinline__ float* at(float* ws, int wg, int slot) { return ws + (2 * wg + slot) * kFloats; }
};

template <int DT, int KIND, int D, int HT>
__global__ __launch_bounds__(256, (kPerCU<KIND, D, HT>)) void attention_kernel(AttentionArgs a) {
    using A = Attend<DT, KIND, D, HT>;
    using Pt = Partial<D, HT>;
    extern __shared__ __align__(16) float lds[];
    __shared__ int s_last;
    A w(a);
    const int lane = w.lane;
    const int wg = blockIdx.x, wgs = gridDim.x;
    const int group = a.group;
    const int head_tiles = (group + A::kCols - 1) / A::kCols;
    const int units = a.H * head_tiles;  // of one sequence

    // Every wave finds the workgroup's share by itself: lane i sums the
    // sequences [i * run, (i + 1) * run), slots above the chunks (which need
    // only be told from more than there are workgroups).
    const int64_t run = (a.B + 63) / 64;
    int64_t sums = 0;
    int length = 0;
    for (int64_t b = lane * run, e = b + run < a.B ? b + run : a.B; b < e; ++b) {
        length = a.lengths[b];
        const int n = Span(a, length).count;
        sums += (int64_t)A::slots_of(n) << kChunkBits;
        if ((sums & kChunkMask) < kChunkMost) sums += chunks_of(n) < kChunkMost ? chunks_of(n) : kChunkMost;
    }
    const int64_t sums_to = wave_scan(sums), all_sums = read_lane(sums_to, 63);
    // Sequences that see nothing.
    for (int64_t b = wg; b < a.B; b += wgs) {
        const int len = run == 1 ? __builtin_amdgcn_readlane(length, (int)b) : a.lengths[b];
        if (Span(a, len).count != 0) continue;
        uint16_t* out = a.out + b * a.o_ts;
        for (int i = threadIdx.x; i < a.H * group * D; i += 256) out[(int64_t)(i / D) * a.o_hs + i % D] = 0;
    }
    // Few tiles: a workgroup per kMinTiles of one head, so that most heads
    // need no join. Else equal runs of the list, across heads; a head takes
    // kHeadCost slots before its tiles' ones.
    int chunk = kMinTiles;
    bool by_chunk = units * (all_sums & kChunkMask) <= wgs;
    int64_t all = units * (by_chunk ? all_sums & kChunkMask : all_sums >> kChunkBits);
    int64_t per = by_chunk ? 1 : (all + wgs - 1) >> __builtin_ctz(wgs);
    int64_t seq_items = by_chunk ? sums & kChunkMask : sums >> kChunkBits;  // of sequence base + lane, when base is found
    int64_t seq_to = by_chunk ? sums_to & kChunkMask : sums_to >> kChunkBits;
    if (!by_chunk && run == 1 && units * a.B < wgs && 16 * units * a.B >= wgs) {
        // Heads that are cut anyway, but in few parts, are cut evenly if that
        // fits: a run across two heads starts and ends twice (64 x 4096 tokens
        // of one kv head, 32 query heads: 36 and 32 us; 4 x 9000 of 8 heads of
        // 256 in int8 39 and 33).
        const int n = Span(a, length).count;
        const int most = (int)per + A::kHeadCost / 2, least = (int)per - A::kHeadCost;
        for (int c = most; c >= kMinTiles && c >= least; c -= A::kHeadCost / 2) {
            const int64_t items = (n + c - 1) / c, to = wave_scan(items);
            if (units * read_lane(to, 63) > wgs) break;
            chunk = c;
            by_chunk = true;
            seq_items = items;
            seq_to = to;
        }
        if (by_chunk) {
            all = units * read_lane(seq_to, 63);
            per = 1;
        }
    }
    int64_t pos = wg * per;
    const int64_t end = pos + per < all ? pos + per : all;
    if (pos >= end) return;

    // The block of 64 sequences that holds `pos`, and in it the sequence.
    int64_t base = 0;
    auto block_at = [&](int64_t first, int64_t before) {  // `before`: items of the sequences before it
        base = first;
        length = base + lane < a.B ? a.lengths[base + lane] : 0;
        const int n = Span(a, length).count;
        seq_items = by_chunk ? chunks_of(n) : A::slots_of(n);
        seq_to = before + wave_scan(seq_items);
    };
    if (run > 1) {
        const int at = __builtin_ctzll(__builtin_amdgcn_ballot_w64(units * seq_to > pos));
        block_at(at * run, read_lane(seq_to - seq_items, at));
        while (units * read_lane(seq_to, 63) <= pos) block_at(base + 64, read_lane(seq_to, 63));
    }
    int at = __builtin_ctzll(__builtin_amdgcn_ballot_w64(units * seq_to > pos));

    while (pos < end) {
        // Sequence b = base + at; its items start at seq_begin.
        const int64_t b = base + at;
        const int items = (int)read_lane(seq_items, at);  // of one unit
        const int64_t seq_end = units * read_lane(seq_to, at), seq_begin = seq_end - (int64_t)units * items;
        const Span sp(a, __builtin_amdgcn_readlane(length, at));
        int unit = divide(pos - seq_begin, items);
        for (; pos < end && pos < seq_end; ++unit) {
            const int64_t unit_begin = seq_begin + (int64_t)unit * items, unit_end = unit_begin + items;
            const int64_t stop = unit_end < end ? unit_end : end;
            int from = (int)(pos - unit_begin), upto = (int)(stop - unit_begin);
            pos = stop;
            if (by_chunk) {
                from *= chunk;
                upto = upto * chunk < sp.count ? upto * chunk : sp.count;
            } else {
                from = from > A::kHeadCost ? from - A::kHeadCost : 0;
                upto -= A::kHeadCost;
                if (upto <= 0) break;  // the head's tiles begin in the next workgroup
            }
            const bool whole = from == 0 && upto == sp.count;
            const int kv_head = head_tiles == 1 ? unit : unit / head_tiles, head_tile = unit - kv_head * head_tiles;
            const int head0 = kv_head * group + head_tile * A::kCols;
            const int heads = group - head_tile * A::kCols < A::kCols ? group - head_tile * A::kCols : A::kCols;

            w.load_query(b, head0, heads);
            w.run(b, kv_head, sp, sp.first + from, sp.first + upto);
            __syncthreads();  // the last join's reads of LDS are done
            w.to_lds(lds, heads);
            __syncthreads();
            const float* ml = lds + kWaves * heads * A::kLd;
            const int slot = from == 0 ? 1 : 0;
            for (int e = threadIdx.x; e < heads * (D / 4); e += 256) {
                const int head = e / (D / 4), d = e % (D / 4) * 4;
                Join j;
#pragma unroll
                for (int v = 0; v < kWaves; ++v) j.m = fmaxf(j.m, ml[2 * (v * heads + head)]);
#pragma unroll
                for (int v = 0; v < kWaves; ++v)
                    j.add(ml[2 * (v * heads + head)], ml[2 * (v * heads + head) + 1],
                          *reinterpret_cast<const floatx4*>(lds + (v * heads + head) * A::kLd + d));
                if (whole) {
                    store_out<DT>(a, b, head0 + head, d, j);
                } else {
                    float* p = Pt::at(a.partials, wg, slot) + head * Pt::kStride;
                    store_coherent(p + 4 + d, j.o);
                    if (d == 0) store_coherent2(p, j.m, j.l);
                }
            }
            if (whole) continue;

            // Join: of kFan workgroups, by the last of them; then of those results.
            const int first = by_chunk ? wg - from / chunk : divide(unit_begin + A::kHeadCost, per);
            const int last = by_chunk ? first + items - 1 : divide(unit_end - 1, per);
            int rank = wg - first, count = last - first + 1, step = 1;
            uint32_t* counters = a.counters;
            for (int level = 0;; ++level) {
                const int lead = rank / kFan * kFan;
                const int size = count - lead < kFan ? count - lead : kFan;
                const int lead_wg = first + lead * step, lead_slot = lead == 0 ? 1 : 0;
                wait_vector_memory();
                __syncthreads();
                if (threadIdx.x == 0) {
                    uint32_t* counter = counters + 2 * lead_wg + lead_slot;
                    const uint32_t old = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    s_last = old + 1 == (uint32_t)size;
                    if (old + 1 == (uint32_t)size) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                }
                __syncthreads();
                const bool mine = s_last != 0;
                if (!mine) break;
                const bool done = count <= kFan;
                const int pair = level & 1 ? 2 : 0;
                float* lead_p = Pt::at(a.partials, lead_wg, lead_slot);
                const float* from[kFan];
#pragma unroll
                for (int i = 0; i < kFan; ++i)
                    from[i] = uniform(i == 0 || size == 1 ? lead_p : Pt::at(a.partials, lead_wg + (i < size ? i : size - 1) * step, 0));
                for (int e = threadIdx.x; e < heads * (D / 4); e += 256) {
                    const int head = e / (D / 4), d = e % (D / 4) * 4;
                    float2 pml[kFan];
                    floatx4 po[kFan];
                    Join j;
                    const uint32_t at4 = (head * Pt::kStride + 4 + d) * 4, at2 = (head * Pt::kStride + pair) * 4;
                    auto add = [&](int most) {
#pragma unroll
                        for (int i = 0; i < most; ++i) j.m = fmaxf(j.m, pml[i].x);
#pragma unroll
                        for (int i = 0; i < most; ++i)
                            if (i < size) j.add(pml[i].x, pml[i].y, po[i]);
                    };
                    if (size <= kFan / 2) {
                        load_coherent8_half(from, at4, at2, po, pml);
                        add(kFan / 2);
                    } else {
                        load_coherent8(from, at4, at2, po, pml);
                        add(kFan);
                    }
                    if (done) {
                        store_out<DT>(a, b, head0 + head, d, j);
                    } else {  // in the leader's place
                        float* p = lead_p + head * Pt::kStride;
                        store_coherent(p + 4 + d, j.o);
                        if (d == 0) store_coherent2(p + (2 - pair), j.m, j.l);
                    }
                }
                if (done) break;
                rank = lead / kFan;
                step *= kFan;
                count = (count + kFan - 1) / kFan;
                counters += 2 * wgs;
            }
        }
        // The next sequence that sees anything.
        if (pos >= end) break;
        uint64_t rest = at < 63 ? __builtin_amdgcn_ballot_w64(seq_items > 0) >> (at + 1) << (at + 1) : 0;
        while (rest == 0) {
            block_at(base + 64, read_lane(seq_to, 63));
            rest = __builtin_amdgcn_ballot_w64(seq_items > 0);
        }
        at = __builtin_ctzll(rest);
    }
}

struct Shape {
    int heads, per_cu;      // query heads of a workgroup's operand, workgroups per CU
    int64_t wgs;
    int64_t partial_floats; // of one workgroup
};

template <int KIND, int D, int HT>
Shape shape_of() {
    return {16 * HT, kPerCU<KIND, D, HT>, 0, 2 * Partial<D, HT>::kFloats};
}

// Calls fn with the head size and the head tiles as constants.
template <class Fn>
void by_shape(int D, int group, Fn&& fn) {
    using std::integral_constant;
    auto with = [&](auto d) {
        if (group <= 16) fn(d, integral_constant<int, 1>{});
        else fn(d, integral_constant<int, 2>{});
    };
    if (D == 64) with(integral_constant<int, 64>{});
    else if (D == 128) with(integral_constant<int, 128>{});
    else if (D == 192) with(integral_constant<int, 192>{});
    else with(integral_constant<int, 256>{});
}

// As many workgroups as run at once, or as there can be parts of kMinTiles.
Shape plan(const AttentionArgs& a, int kind) {
    Shape s{};
    const int group = a.Hq / a.H;
    by_shape(a.D, group, [&](auto d, auto ht) {
        s = kind == 0 ? shape_of<0, decltype(d)::value, decltype(ht)::value>() : shape_of<1, decltype(d)::value, decltype(ht)::value>();
    });
    int64_t tokens = a.width * a.P;
    if (a.window > 0 && a.window < tokens) tokens = a.window + kTile;
    const int64_t parts = (tokens / kTile + kMinTiles) / kMinTiles;
    const int64_t units = (int64_t)a.H * ((group + s.heads - 1) / s.heads);
    s.wgs = kCUs * s.per_cu;
    if (a.B * units < s.wgs && a.B * units * parts < s.wgs) s.wgs = a.B * units * parts;
    return s;
}

template <int DT, int KIND>
hipError_t launch(const AttentionArgs& a, const Shape& s, hipStream_t stream) {
    hipError_t e = hipSuccess;
    const int group = a.Hq / a.H;
    by_shape(a.D, group, [&](auto d, auto ht) {
        constexpr int D = decltype(d)::value, HT = decltype(ht)::value;
        const int heads = group < 16 * HT ? group : 16 * HT;
        const size_t lds = (size_t)kWaves * heads * (Attend<DT, KIND, D, HT>::kLd + 2) * 4;
        e = allow_lds<attention_kernel<DT, KIND, D, HT>>(lds);
        if (e != hipSuccess) return;
        hipLaunchKernelGGL((attention_kernel<DT, KIND, D, HT>), dim3((unsigned)s.wgs), dim3(256), lds, stream, a);
        e = hipGetLastError();
    });
    return e;
}

}  // namespace

size_t attention_workspace(const AttentionArgs& a, int kind) {
    const Shape s = plan(a, kind);
    return kCounterRegionBytes + (size_t)s.wgs * s.partial_floats * 4;
}

hipError_t launch_attention(AttentionArgs a, int kind, int dtype, void* workspace, hipStream_t stream) {
    const Shape s = plan(a, kind);
    a.group = a.Hq / a.H;
    const int64_t most = a.width * a.P, all = ((int64_t)1 << 31) - 1;
    a.most = (int)(most < all ? most : all);
    a.reach = (int)(a.window > 0 && a.window < all ? a.window : all);
    a.counters = static_cast<uint32_t*>(workspace);
    a.partials = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + kCounterRegionBytes);
    if (kind == 0) return dtype == 0 ? launch<0, 0>(a, s, stream) : launch<1, 0>(a, s, stream);
    return dtype == 0 ? launch<0, 1>(a, s, stream) : launch<1, 1>(a, s, stream);
}

}  // namespace w4a16
