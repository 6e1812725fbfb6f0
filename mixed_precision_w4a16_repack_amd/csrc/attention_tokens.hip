// attention_tokens.hip -- attention of several new tokens per sequence over
// the paged key/value cache (prompts, chunks of them, trees of drafted tokens):
//   s_t = scale * q . k_t,  o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),
// over the tokens t that a row sees, in one pass: sums and output are relative to
// 2^r of a reference r that moves only when a score passes it by 2^2 (fp16) or
// 2^8 (bf16), so that most tiles multiply nothing again.
//
// A block is 64 or 128 rows (token, query head of one kv head, heads fastest) of
// a sequence: the rows of a kv head share its tiles. Four waves take 16 or 32 rows
// each, as columns: S^T = K Q^T leaves the scores of 4 tokens of one row in a lane,
// which are P^T's operand of O^T += V^T P^T as they are; the cache's tiles are
// both products' other operands as stored. A probability is two 16-bit operands, its
// rounding and the rest's (over int8 with bf16 results one fp16 operand, an eighth
// of the result's half step), sums, references and outputs are fp32.
//
// Tiles of 32 tokens come straight into a ring of 3 or 4 places in LDS, two ahead, by
// loads that the waits count: every wave loads the same number of pieces for each tile, in
// order, and what else it loads only makes a wait longer. int8 tiles are
// turned into fp16 operands once a block, keys two tiles ahead and values one, and
// their scales go into the scores and the probabilities. One barrier a tile. A tile's
// products are made before its turn, between the exponentials of the tile
// before, in written order: left to the compiler they came apart, and
// prompts took 7 % more.
//
// Blocks differ in length (causal, ragged), so the list of all blocks' tiles is
// cut into equal runs, one a workgroup, from the lengths, on the device; a
// block that lies in several leaves partial results, which a second kernel joins.
//
// What bounds it: the SIMDs' instructions. A wave's step of 32 rows and 32 tokens is 48
// matrix products (16 cycles each), 180 other vector instructions (16 of them
// exponentials) and 68 scalar ones; the matrix cores are busy for 42 % of the time and the
// other vector instructions take as much again, and the two waves of a SIMD overlap little of it:
// without the products, the exponentials or the loads the time falls by about that part's own.
// Four prompts of 2048 tokens, 32 heads of 128 over 8, bf16: 229 us a call, 601 TFLOP/s
// (the two-operand products counted once; 222 to 237 between boxes and ways of timing); 24
// trees of 32 tokens over up to 6000: 80 us; two trees of 80 tokens over 50000 of int8, 64
// heads: 432 us, 606 TFLOP/s; one tree of 16 tokens over 700: 20 us, of which 4 find the
// share and 4 join.
// Columns of 64 rows a wave with one workgroup a CU: 702 us for the 255 of then.
#include <cmath>

#include "attention_common.h"
#include "device_common.h"
#include "internal.h"
#include "kv_layout.h"
#include "lds_stage.h"

namespace w4a16 {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;       // tokens
// A block's start and end cost about as much as this many tiles (with 3: prompts 284 us
// for 275, short trees 99 for 85; with 10: 283 and 85).
constexpr int kHeadTiles = 6;
// A workgroup's least share beside that: a split costs a part of a join (one tree of
// 16 tokens with 3, 5 and 8: 22.7, 23.3 and 25.3 us).
constexpr int kLeastTiles = 3;

// What the rows of a block see together: tokens lo .. hi - 1 and 0 .. sk - 1
// (sk <= lo), in `count` tiles: `head` of them before the window's, which lie
// `skip` tiles further on.
struct Span {
    int lo, hi, sk, head, skip, count;
    __device__ __forceinline__ int tile(int i) const { return i < head ? i : i + skip; }
};

// A sequence: n tokens in the cache, the last m of them new, in rows from `row` on.
struct Sequence {
    int64_t row;
    int m, n;
    __device__ __forceinline__ Sequence() : row(0), m(0), n(0) {}
    __device__ __forceinline__ Sequence(const TokensArgs& a, int64_t b) {
        const int64_t from = a.starts[b], to = a.starts[b + 1];
        row = from < 0 ? 0 : (from < a.T ? from : a.T);
        const int64_t end = to < row ? row : (to < a.T ? to : a.T);
        m = (int)(end - row);
        const int len = a.lengths[b];
        n = len < 0 ? 0 : (len > a.most ? a.most : len);
    }
};

template <int ROWS>
struct Blocks {
    // Rows of a block: (token, query head of the group), heads fastest.
    static __device__ __forceinline__ int count(const TokensArgs& a, int m) {
        return (int)(((int64_t)m * a.group + ROWS - 1) / ROWS);
    }
    static __device__ __forceinline__ Span span(const TokensArgs& a, int m, int n, int j) {
        const uint32_t first = (uint32_t)j * ROWS;  // rows are counted in 31 bits
        const int i0 = a.token_of(first), to = a.token_of(first + ROWS - 1), i1 = to < m ? to : m - 1;
        Span s;
        const int64_t past = (int64_t)n - m;  // may be negative: new tokens that have no place see nothing
        const int64_t hi = a.tree ? n : past + i1 + 1;
        const int64_t at = a.tree ? past : past + i0;  // the first row's position
        const int64_t lo = at + 1 - a.reach;
        s.hi = hi > 0 ? (int)hi : 0;
        s.lo = lo > 0 ? (int)lo : 0;
        s.sk = a.sinks < s.lo ? a.sinks : s.lo;
        const int window = s.lo / kTile, tiles = (s.sk + kTile - 1) / kTile;
        s.head = tiles < window ? tiles : window;
        s.skip = window - s.head;
        s.count = s.hi > s.lo ? (s.hi - 1) / kTile + 1 - s.skip : 0;
        return s;
    }
    static __device__ __forceinline__ int cost(const TokensArgs& a, int m, int n, int j) { return span(a, m, n, j).count + kHeadTiles; }
};

typedef short short2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t below(int64_t x) { return x <= 0 ? 0u : (x >= 32 ? ~0u : (1u << x) - 1u); }

// A value that is the same on all lanes, so that branches on it are not masked.
__device__ __forceinline__ int same(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t same(int64_t x) { return read_lane(x, 0); }

// N pieces of 1024 bytes from a buffer straight into LDS, 16 bytes a lane. In
// asm, so that the compiler does not wait for them at every LDS read: the ring's
// own waits do (wait_vmcnt, then the barrier). They only make the compiler's other
// waits stricter. s_nop: the descriptor may come from a VALU instruction (5
// wait states to the load), M0 needs one. M0 is reserved and cannot be named as
// changed: the build checks that the compiler itself uses it in none of these kernels.
template <int N>
__device__ __forceinline__ void load_lds(const u32x4& rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
    static_assert(N >= 1, "pieces");
    if constexpr (N >= 4) {
        asm volatile(
            "s_nop 4\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\t"
            "buffer_load_dwordx4 %1, %2, %3 offen lds\n\t"
            "buffer_load_dwordx4 %1, %2, %3 offen offset:1024 lds\n\t"
            "buffer_load_dwordx4 %1, %2, %3 offen offset:2048 lds\n\t"
            "buffer_load_dwordx4 %1, %2, %3 offen offset:3072 lds" ::"s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
            : "memory");
        if constexpr (N > 4) load_lds<N - 4>(rsrc, lds + 4096, voff, soff + 4096);
    } else if constexpr (N >= 2) {
        asm volatile(
            "s_nop 4\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\t"
            "buffer_load_dwordx4 %1, %2, %3 offen lds\n\t"
            "buffer_load_dwordx4 %1, %2, %3 offen offset:1024 lds" ::"s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
            : "memory");
        if constexpr (N > 2) load_lds<N - 2>(rsrc, lds + 2048, voff, soff + 2048);
    } else {
        asm volatile("s_nop 4\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
                     "s"(rsrc), "s"(soff)
                     : "memory");
    }
}
// 4 bytes a lane.
__device__ __forceinline__ void load_lds_words(const u32x4& rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
    asm volatile("s_nop 4\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(lds), "v"(voff), "s"(rsrc),
                 "s"(soff)
                 : "memory");
}

// A workgroup's part of a block: items [from, upto) of its tiles.
struct Item {
    int64_t b, row;
    int m, n, kv_head, j, from, upto;
    int parts;  // workgroups that share the block, if it begins here and does not end here
    int whole;  // it begins and ends here
};
constexpr int kItems = 24;  // found at once, in LDS

template <int DT, int KIND, int D, int HT>
struct Attend {
    static constexpr bool kI8 = KIND == 1;
    static constexpr bool kF16P = kI8 || DT == 0;
    static constexpr int PDT = kF16P ? 0 : 1;          // operand type of both products
    static constexpr int NP = kI8 && DT == 1 ? 1 : 2;  // operands of a probability
    static constexpr int NQ = D / 32;                  // MFMAs along d
    static constexpr int NO = D / 16;
    static constexpr int kRows = 16 * HT * kWaves;
    // A tile as loaded: keys, then values, kLoads pieces of 1024 bytes a wave;
    // int8: codes, then key scales and value scales.
    static constexpr int kLoads = 2 * D * (kI8 ? 1 : 2) * kTile / 1024 / kWaves;
    static constexpr int kRaw = kLoads * kWaves * 1024 + (kI8 ? 256 : 0);
    static constexpr int kTileLoads = kLoads + (kI8 ? 1 : 0);
    // Operands of a tile's keys, and of its values: 16 bits each. 16-bit tiles
    // are operands as loaded; int8 ones are turned into them, in two places for
    // keys, two for values and three for scales.
    static constexpr int kPart = D * kTile * 2;
    static constexpr int kOperands = kI8 ? 4 * kPart + 3 * 256 : 0;
    // Workgroups that share a CU, and tiles in the ring that loads fill.
    static constexpr int kListed = 128;  // tiles in hand: 64 found at once, and a few not yet worked on
    static constexpr int kPerCU = D <= 128 || (D == 192 && HT == 1 && !kI8) ? 2 : 1;
    static constexpr int kFree = (kPerCU == 2 ? 80 : 160) * 1024 - kItems * (int)sizeof(Item) - (kListed + 1) * 16 - kOperands;
    static constexpr int kStages = kFree / kRaw < 4 ? kFree / kRaw : 4;
    static constexpr int kBytes = kStages * kRaw + kOperands + (kListed + 1) * 16 + kItems * (int)sizeof(Item);
    static_assert(kStages >= 3, "a tile is loaded while others are worked on");
    using L = KvPlace<KIND>;
    using Pr = Prob<kF16P>;

    const TokensArgs& a;
    unsigned char* lds;
    const int lane, wave, g, col;
    u32x4 q[HT][NQ];
    float factor[HT];
    floatx4 o[HT][NO];
    float r[HT], l[HT];
    static constexpr float kFar = 96.0f;  // int8: sums of 2^31 probabilities of 2^kFar, 2^127, are within fp32
    // Of each column: what it sees, tokens lo .. hi - 1 and 0 .. sk - 1, and tree bits from `past` on.
    int lo[HT], hi[HT];
    int64_t row;   // of the block's sequence
    int past, first, rows;  // tokens before the new ones (may be negative), the block's first row and the sequence's rows
    int full_lo, full_hi;   // tiles in [full_lo, full_hi) are seen whole by every column of the wave
    bool busy;     // the wave has a row

    __device__ __forceinline__ Attend(const TokensArgs& args, unsigned char* smem)
        : a(args), lds(smem), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), g(lane >> 4), col(lane & 15) {}

    // Row (token of the sequence's new ones, query head of the group) of column h.
    __device__ __forceinline__ int row_at(int h) const { return first + (wave * HT + h) * 16 + col; }

    __device__ __forceinline__ void begin(const Item& it) {
        const int kv_head = it.kv_head;
        past = it.n - it.m;
        row = it.row;
        first = it.j * kRows;
        rows = it.m * a.group;
        busy = same(first + wave * HT * 16) < same(rows);
        int least_hi = 0x7FFFFFFF, most_lo = 0;
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            const int at_row = row_at(h), i = a.token_of(at_row), head = kv_head * a.group + at_row - i * a.group;
            lo[h] = 0;
            hi[h] = 0x7FFFFFFF;  // columns without a row do not count
            if (at_row < rows) {
                int at = past + i, end = at + 1;
                if (a.tree) {
                    int depth = 0;  // set bits of the it.m new tokens: those behind them stand for no token
                    uint64_t any = 0;
                    for (int w = 0; w < a.tree_words; ++w) {
                        const uint64_t word = a.tree[(row + i) * a.tree_ld + w];
                        const int left = it.m - 64 * w;
                        depth += __builtin_popcountll(left >= 64 ? word : (left > 0 ? word & (((uint64_t)1 << left) - 1) : 0));
                        any |= word;
                    }
                    at = past + (depth > 0 ? depth - 1 : 0);
                    end = any != 0 ? past : 0;  // past tokens; the tree's by their bits
                }
                hi[h] = end > 0 ? end : 0;
                lo[h] = at >= a.reach ? (int)(at + 1 - a.reach) : 0;
            }
            least_hi = hi[h] < least_hi ? hi[h] : least_hi;
            most_lo = lo[h] > most_lo ? lo[h] : most_lo;
            const uint16_t* p = a.q + (row + i) * a.q_ts + (int64_t)head * a.q_hs + 8 * g;
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                q[h][x] = u32x4{0u, 0u, 0u, 0u};
                if (at_row < rows) q[h][x] = *reinterpret_cast<const u32x4_any*>(p + 32 * x);
            }
            r[h] = kLowest;
            l[h] = 0.0f;
#pragma unroll
            for (int x = 0; x < NO; ++x) o[h][x] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int off = 1; off < 16; off *= 2) {
            const int x = __shfl_xor(least_hi, off), y = __shfl_xor(most_lo, off);
            least_hi = x < least_hi ? x : least_hi;
            most_lo = y > most_lo ? y : most_lo;
        }
        full_hi = __builtin_amdgcn_readfirstlane(least_hi);
        full_lo = __builtin_amdgcn_readfirstlane(most_lo);
        convert_query();
    }

    // A negative scale's sign goes into the queries, and a scale of 0 (so that a
    // factor on an unseen score of -infinity is positive): the largest product
    // has the largest score. bf16 queries over int8 are moved by a power of two to the
    // top of fp16's range.
    __device__ __forceinline__ void convert_query() {
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u, keep = a.scale == 0.0f ? 0u : ~0u;
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            factor[h] = a.scale == 0.0f ? 1.0f : __builtin_fabsf(a.scale) * 1.44269504088896341f;
#pragma unroll
            for (int i = 0; i < NQ; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) q[h][i][e] = (q[h][i][e] ^ flip) & keep;
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
                const int e = (int)(top >> 7);  // biased exponent of the row's largest element
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
                // Never 0, which times an unseen score's -infinity is NaN: the least number in its
                // place moves a score by less than 2^-21, since products are below 2^128.
                factor[h] = __builtin_ldexpf(factor[h], -up);
                if (factor[h] == 0.0f) factor[h] = 0x1p-149f;
            }
        }
    }

    // This wave's part of a tile on its way to a place of the ring: half the waves load keys, half values.
    __device__ __forceinline__ void request(uint64_t at, int sub, int place) {
        constexpr uint32_t kKeys = kLoads * kWaves / 2 * 1024;  // bytes of a tile's keys, and of its values
        const u32x4 rsrc{(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, (uint32_t)L::record_bytes(D, a.P), 0x00020000u};
        const uint32_t to = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)lds + place * kRaw);
        const uint32_t part = (uint32_t)(wave % (kWaves / 2)) * kLoads * 1024;
        const uint32_t from = (wave < kWaves / 2 ? 0u : (uint32_t)L::keys_bytes(D, a.P)) + (uint32_t)sub * kKeys + part;
        load_lds<kLoads>(rsrc, to + wave * kLoads * 1024, lane * 16, from);
        // Every wave loads the scales, the same ones: as many loads a wave.
        if constexpr (kI8)
            load_lds_words(rsrc, to + kLoads * kWaves * 1024, (lane & 31) * 4 + (lane < 32 ? 0 : a.P * 4),
                           (uint32_t)(2 * L::keys_bytes(D, a.P)) + sub * kTile * 4);
    }
    // Where a tile's operands and scales are: 16 bits, in the ring; int8, tile i's in place i % 2, scales in i % 3.
    __device__ __forceinline__ const unsigned char* keys_at(int place, int i) const { return lds + (kI8 ? kStages * kRaw + (i & 1) * kPart : place * kRaw); }
    __device__ __forceinline__ const unsigned char* values_at(int place, int i) const {
        return lds + (kI8 ? kStages * kRaw + (2 + (i & 1)) * kPart : place * kRaw + kPart);
    }
    __device__ __forceinline__ const float* scales_at(int third) const {
        return reinterpret_cast<const float*>(lds + kStages * kRaw + 4 * kPart + third * 256);
    }
    // int8: this wave's part of a tile in the ring, and as operands of tile i; half the waves turn keys, half values.
    __device__ __forceinline__ void read_codes(int place, u32x4 (&v)[kLoads]) const {
        const u32x4* from = reinterpret_cast<const u32x4*>(lds + place * kRaw) + wave * kLoads * 64 + lane;
#pragma unroll
        for (int x = 0; x < kLoads; ++x) v[x] = from[64 * x];
    }
    __device__ __forceinline__ void convert(const u32x4 (&v)[kLoads], int i) {
        const unsigned char* part = wave < kWaves / 2 ? keys_at(0, i) : values_at(0, i);
        u32x4* to = reinterpret_cast<u32x4*>(const_cast<unsigned char*>(part)) + wave % (kWaves / 2) * kLoads * 128 + lane;
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
            to[128 * x] = codes8_to_f16(v[x][0], v[x][1]);
            to[128 * x + 64] = codes8_to_f16(v[x][2], v[x][3]);
        }
    }
    __device__ __forceinline__ void copy_scales(int place, int third) {
        if (wave == 0) const_cast<float*>(scales_at(third))[lane] = reinterpret_cast<const float*>(lds + place * kRaw + kLoads * kWaves * 1024)[lane];
    }

    // Which of the tile's 32 tokens column h sees.
    __device__ __forceinline__ uint32_t visible(int h, int at, int n) const {
        uint32_t seen = below(hi[h] - at) & (~below(lo[h] - at) | below((a.sinks < lo[h] ? a.sinks : lo[h]) - at));
        if (same((int)(a.tree != nullptr && at + (int64_t)kTile > past)) != 0) {  // no branch that lanes take differently
            const int at_row = row_at(h);
            const int64_t bit = (int64_t)at - past;  // of the tile's first token
            const uint64_t* words = a.tree + (row + a.token_of(at_row < rows ? at_row : rows - 1)) * a.tree_ld;
            uint32_t bits = 0u;
            if (same((int)(bit < 0)) != 0) {
                bits = (uint32_t)(words[0] << -bit);
            } else if (same((int)(bit < 64 * (int64_t)a.tree_words)) != 0) {
                const int w = (int)(bit >> 6), by = (int)(bit & 63);
                const int next = w + 1 < a.tree_words ? w + 1 : w;
                const uint64_t more = next > w && by > 32 ? words[next] << (64 - by) : 0u;
                bits = (uint32_t)(words[w] >> by | more);
            }
            seen |= at_row < rows ? bits & below(n - at) : 0u;
        }
        return seen;
    }

    // s[h][0][..]: tokens 4g .. 4g+3 of a tile, s[h][1][..]: 16 tokens on.
    __device__ __forceinline__ void products(const unsigned char* keys, floatx4 (&s)[HT][2]) const {
        const u32x4* tile = reinterpret_cast<const u32x4*>(keys) + lane;
#pragma unroll
        for (int h = 0; h < HT; ++h)
#pragma unroll
            for (int t = 0; t < 2; ++t) s[h][t] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const u32x4 k = tile[(t * NQ + i) * 64];
#pragma unroll
                for (int h = 0; h < HT; ++h) s[h][t] = mfma16x16x32<PDT>(k, q[h][i], s[h][t]);
            }
    }

    // All bits of the halves of a word that hold finite numbers.
    static __device__ __forceinline__ uint32_t finite(uint32_t pair) {
        constexpr uint32_t kInf = DT == 0 ? 0x7C007C00u : 0x7F807F80u;
        const short2_t x = __builtin_bit_cast(short2_t, pair & kInf) - __builtin_bit_cast(short2_t, kInf);
        return __builtin_bit_cast(uint32_t, x >> 15);
    }

    // int8: scores from a tile's products, and its values' scales.
    __device__ __forceinline__ void apply_scales(const float* scales, floatx4 (&s)[HT][2], floatx4 (&vs)[2]) const {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const floatx4 ks = *reinterpret_cast<const floatx4*>(scales + 4 * g + 16 * t);
            vs[t] = *reinterpret_cast<const floatx4*>(scales + 32 + 4 * g + 16 * t);
#pragma unroll
            for (int h = 0; h < HT; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[h][t][e] *= ks[e];
        }
    }
    __device__ __forceinline__ float largest(const floatx4 (&s)[2]) const {
        float x = s[0][0];
#pragma unroll
        for (int j = 1; j < 8; ++j) x = fmaxf(x, s[j / 4][j % 4]);
        return x;
    }
    // Above 0: a score is so far above its column's reference r that this has to
    // move. Sums are relative to 2^r, which keeps the largest weight (a probability,
    // int8 times the value's scale) within the operand's range.
    __device__ __forceinline__ float above(const floatx4 (&s)[HT][2], const floatx4 (&vs)[2]) const {
        float more = 0.0f;  // int8: log2 of the largest scale of the lane's values
        if constexpr (kI8) more = __builtin_amdgcn_logf(fmaxf(largest(vs), 0.0f));
        float by = kLowest;
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            const float peak = largest(s[h]) * factor[h];
            by = fmaxf(by, peak + more - (r[h] + (Pr::kBias + Pr::kHeadroom)));
            if constexpr (kI8) by = fmaxf(by, peak - (r[h] + kFar));
        }
        return by;
    }

    // A tile of tokens from `at` on, whose scores s holds (before the scale's
    // factor), `over` above()'s answer; whole: every column sees all of them. The next
    // tile's products and answer are made on the way, so that the matrix cores have work
    // while the probabilities are formed, and nothing waits for the answer.
    __device__ __forceinline__ void work(floatx4 (&s)[HT][2], floatx4 (&vs)[2], float& over, const unsigned char* next_keys,
                                         const float* next_scales, const unsigned char* operands, int at, int n, bool whole) {
        __builtin_amdgcn_s_setprio(0);
        u32x4 v[NO];
#pragma unroll
        for (int i = 0; i < NO; ++i) v[i] = reinterpret_cast<const u32x4*>(operands)[64 * i + lane];
        uint32_t seen[HT];
        if (same((int)whole) == 0) {
            // Unseen scores are -infinity. An unseen value may be anything, and
            // 0 * NaN is NaN: an int8 value's scale that is not finite gives way
            // to a score of NaN in the columns that see it.
#pragma unroll
            for (int h = 0; h < HT; ++h) {
                const uint32_t bits = visible(h, at, n);
                seen[h] = (bits >> (4 * g) & 0xFu) | (bits >> (16 + 4 * g) & 0xFu) << 4;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t mask = (uint32_t)((int32_t)(seen[h] << (31 - j)) >> 31);
                    float x = s[h][j / 4][j % 4];
                    if constexpr (kI8) x = __builtin_fabsf(vs[j / 4][j % 4]) < INFINITY ? x : NAN;
                    s[h][j / 4][j % 4] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x) & mask) | (0xFF800000u & ~mask));
                }
            }
            if constexpr (kI8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) vs[j / 4][j % 4] = __builtin_fabsf(vs[j / 4][j % 4]) < INFINITY ? vs[j / 4][j % 4] : 0.0f;
            } else {
                uint32_t all = ~0u;
#pragma unroll
                for (int i = 0; i < NO; ++i) {
                    const u32x4 x = v[i];
                    all &= finite(x[0]) & finite(x[1]) & finite(x[2]) & finite(x[3]);
                }
                if (same((int)(__builtin_amdgcn_ballot_w64(all != ~0u) != 0)) != 0) {
                    // Values that are not finite are taken out of the product, and the
                    // columns that see one become NaN there, and stay so.
                    constexpr uint32_t kOne = DT == 0 ? 0x3C003C00u : 0x3F803F80u;
                    u32x4 ones[HT];
#pragma unroll
                    for (int h = 0; h < HT; ++h)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            ones[h][x] = ((seen[h] >> (2 * x) & 1u) | (seen[h] >> (2 * x + 1) & 1u) << 16) * (kOne & 0xFFFFu);
#pragma unroll
                    for (int i = 0; i < NO; ++i) {
                        __builtin_amdgcn_sched_barrier(0);  // one after the other: this is rare, and its registers are everybody's
                        const u32x4 was = v[i], keep{finite(was[0]), finite(was[1]), finite(was[2]), finite(was[3])};
                        const u32x4 is = ~keep & kOne;
                        v[i] = was & keep;
#pragma unroll
                        for (int h = 0; h < HT; ++h) {
                            const floatx4 hits = mfma16x16x32<PDT>(is, ones[h], floatx4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                            for (int r = 0; r < 4; ++r) o[h][i][r] = hits[r] > 0.0f ? NAN : o[h][i][r];
                        }
                    }
                }
            }
            over = above(s, vs);
        }
        if (same((int)(__builtin_amdgcn_ballot_w64(over > 0.0f) != 0)) != 0) {  // rare after the first tiles
#pragma unroll
            for (int h = 0; h < HT; ++h) {
                const float peak = largest(s[h]) * factor[h];
                float up = peak - Pr::kBias;
                if constexpr (kI8) {  // no further below a score than kFar, however small the scales are
                    float y = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        y = fmaxf(y, exp2_fast(__builtin_fmaf(s[h][j / 4][j % 4], factor[h], -peak)) * vs[j / 4][j % 4]);
                    up = fmaxf(peak + __builtin_amdgcn_logf(y) - Pr::kBias, peak - kFar);
                }
                const float to = column_max(fmaxf(r[h], up)), keep = exp2_fast(r[h] - to);
                r[h] = to;
                l[h] *= keep;
#pragma unroll
                for (int i = 0; i < NO; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[h][i][e] *= keep;
            }
        }
        // The next tile's products take turns with the first column tile's
        // probabilities, and a column tile's sums with the next one's.
        floatx4 ahead[HT][2];
        u32x4 p[HT][NP];
        float w[2];
        auto probability = [&](int h, int j) {
            w[j % 2] = exp2_fast(__builtin_fmaf(s[h][j / 4][j % 4], factor[h], -r[h]));
            l[h] += w[j % 2];
            if constexpr (kI8) w[j % 2] *= vs[j / 4][j % 4];
            if (j % 2 == 1) {
                uint32_t parts[NP];
                split_pair<PDT, NP>(w[0], w[1], parts);
#pragma unroll
                for (int i = 0; i < NP; ++i) p[h][i][j / 2] = parts[i];
            }
        };
        constexpr int kKeys = 2 * NQ, kInHand = 4;
        constexpr int kShare = (8 + kKeys - 1) / kKeys, kSums = (NO * NP + 7) / 8;  // of a turn
        const u32x4* tile = reinterpret_cast<const u32x4*>(next_keys) + lane;
        auto key_at = [&](int i) { return tile[(i % 2 * NQ + i / 2) * 64]; };
        u32x4 k[kInHand];
#pragma unroll
        for (int i = 0; i < kInHand; ++i) k[i] = key_at(i);
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
#pragma unroll
            for (int h = 0; h < HT; ++h)
                ahead[h][i % 2] = mfma16x16x32<PDT>(k[i % kInHand], q[h][i / 2], i < 2 ? floatx4{0.0f, 0.0f, 0.0f, 0.0f} : ahead[h][i % 2]);
            if (i + kInHand < kKeys) k[i % kInHand] = key_at(i + kInHand);
#pragma unroll
            for (int j = 0; j < kShare; ++j)
                if (i * kShare + j < 8) probability(0, i * kShare + j);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int h = 0; h < HT; ++h)
#pragma unroll
            for (int x = 0; x < 8; ++x) {
#pragma unroll
                for (int y = 0; y < kSums; ++y) {
                    const int i = x * kSums + y;
                    if (i < NO * NP) o[h][i % NO] = mfma16x16x32<PDT>(v[i % NO], p[h][i / NO], o[h][i % NO]);
                }
                if (h + 1 < HT) probability(h + 1, x);
                else if (x == 0) {
#pragma unroll
                    for (int y = 0; y < HT; ++y)
#pragma unroll
                        for (int t = 0; t < 2; ++t) s[y][t] = ahead[y][t];
                    if constexpr (kI8) apply_scales(next_scales, s, vs);
                    over = above(s, vs);
                }
                if (h + 1 < HT) __builtin_amdgcn_sched_barrier(0);
            }
    }

    // Items [from, to) of the block's tiles, those of missing pages left out.
    __device__ __forceinline__ void run(const Item& it, const Span& sp) {
        const int64_t b = it.b;
        const int kv_head = it.kv_head, n = it.n, to = it.upto;
        const int tiles_per_page = a.P / kTile;
        const int whole_shift = (tiles_per_page & (tiles_per_page - 1)) == 0 ? __builtin_ctz(tiles_per_page) : -1;
        // The tiles that are there, 64 items looked at at once: where each lies
        // (two words), its number in the page, its first token. Every wave writes
        // the same list and reads what it wrote.
        u32x4* list = reinterpret_cast<u32x4*>(lds + kStages * kRaw + kOperands);
        int next_item = it.from, found = 0;
        auto look = [&]() {
            // No branch that lanes take differently: one here makes the compiler keep two copies of the sums.
            const int item = next_item + lane, tile = sp.tile(item < to ? item : to - 1);
            const int i = whole_shift >= 0 ? tile >> whole_shift : tile / tiles_per_page, sub = tile - i * tiles_per_page;
            const int64_t page = a.table[b * a.table_ld + i];
            const bool ok = item < to && page >= 0 && page < a.pages;
            const uint64_t mask = __builtin_amdgcn_ballot_w64(ok);
            const int at = found + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
            const uint64_t place = reinterpret_cast<uint64_t>(a.cache) + (uint64_t)((page * a.H + kv_head) * L::record_bytes(D, a.P));
            list[ok ? at % kListed : kListed] = u32x4{(uint32_t)place, (uint32_t)(place >> 32), (uint32_t)sub, (uint32_t)tile * kTile};
            found = same(found + __builtin_popcountll(mask));
            next_item += 64;
        };
        // The ring: tile i of the list lies in place i % kStages.
        int there = 0, done = 0;  // tiles requested and worked on
        int fill = 0, take = 0;   // their places
        auto list_more = [&]() {  // so that an entry is there for the next request, if any is left
            while (there == found && next_item < to) look();
        };
        auto request_listed = [&](const u32x4& e) {  // e: list[there % kListed]
            request((uint64_t)(uint32_t)same((int)e[1]) << 32 | (uint32_t)same((int)e[0]), same((int)e[2]), fill);
            fill = fill + 1 < kStages ? fill + 1 : 0;
            ++there;
            list_more();
        };
        list_more();
        stage_barrier();  // the ring is free
        // Tile i is worked on when its values and tile i + 1's keys are there.
        // 16 bits: tiles up to i + kStages - 2 are on their way, and when all waves
        // have begun tile i, tile i - 1's place takes tile i + kStages - 1. int8: up to
        // i + kStages - 1; keys become operands two tiles ahead, values one, and the place
        // that takes tile i + kStages is tile i's own.
        constexpr int kAhead = kI8 ? kStages : kStages - 1;
        while (there < found && there < kAhead) request_listed(list[there % kListed]);
        begin(it);  // the queries are on their way too
        if (there == 0) return;
        floatx4 s[HT][2];
        int third = 0;  // int8: the scales' place
        auto place_of = [&](int i) { return i < kStages ? i : i - kStages; };  // take + i
        auto wait_for = [&](int younger) {  // until at most that many tiles are on their way
            if (younger >= 2) wait_vmcnt<2 * kTileLoads>();
            else if (younger == 1) wait_vmcnt<kTileLoads>();
            else wait_vmcnt<0>();
        };
        if constexpr (kI8) {
            wait_for(there - 2 < 0 ? 0 : there - 2);
            stage_barrier();
            u32x4 codes[kLoads];
            read_codes(0, codes);
            convert(codes, 0);
            copy_scales(0, 0);
            if (there > 1) {
                if (wave < kWaves / 2) {
                    read_codes(1, codes);
                    convert(codes, 1);
                }
                copy_scales(1, 1);
            }
            stage_barrier();
        } else {
            wait_for(there - 1);
            stage_barrier();
        }
        floatx4 vs[2];
        float over = 0.0f;
        if (busy) {
            products(keys_at(0, 0), s);
            if constexpr (kI8) apply_scales(scales_at(0), s, vs);
            over = above(s, vs);
        }
        // The next tile to work on: its first token, its place and the next one's.
        int t = 0, place = 0, next = 0;
        // A wave between two tiles goes before the CU's others, which the next barrier
        // or its next loads wait for (3 % of the time of prompts, 4 % of long int8 ones).
        auto advance = [&]() -> bool {
            __builtin_amdgcn_s_setprio(3);
            if (done == there) return false;
            // Read before the wait, needed behind it.
            const u32x4 e = list[there % kListed];
            const uint32_t first_token = reinterpret_cast<const uint32_t*>(list)[done % kListed * 4 + 3];
            place = take;
            next = place_of(take + 1);
            const int left = there - done;  // this one, the ones that are there and the ones on their way
            wait_for(left - (kI8 ? 3 : 2) < 0 ? 0 : left - (kI8 ? 3 : 2));
            stage_barrier();
            u32x4 codes[kLoads];
            // int8: into places that were read for tile done - 1, or before.
            const bool turns = kI8 && left > (wave < kWaves / 2 ? 2 : 1);
            const int from = place_of(take + (wave < kWaves / 2 ? 2 : 1));
            if (kI8 && turns) read_codes(from, codes);
            t = same((int)first_token);
            if (there < found) request_listed(e);
            if constexpr (kI8) {
                if (turns) convert(codes, done + (wave < kWaves / 2 ? 2 : 1));
                if (left > 2) copy_scales(place_of(take + 2), third >= 1 ? third - 1 : 2);
                third = third < 2 ? third + 1 : 0;  // the next tile's
            }
            take = next;
            ++done;
            return true;
        };
        auto whole = [&]() { return t <= full_hi - kTile && (t >= full_lo || t <= a.sinks - kTile); };
        bool have = advance();
        if (!busy) {
            while (have) have = advance();
            return;
        }
        while (have) {
            work(s, vs, over, keys_at(next, done), scales_at(third), values_at(place, done - 1), t, n, whole());
            have = advance();
        }
    }

    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int h = 0; h < HT; ++h) l[h] = column_sum(l[h]);
    }
    __device__ __forceinline__ void store_out(int kv_head) {
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            const int at_row = row_at(h), t = a.token_of(at_row);
            if (at_row >= rows) continue;
            const float inv = 1.0f / (l[h] == 0.0f ? 1.0f : l[h]);
            uint16_t* out = a.out + (row + t) * a.o_ts + (int64_t)(kv_head * a.group + at_row - t * a.group) * a.o_hs + 4 * g;
#pragma unroll
            for (int i = 0; i < NO; ++i) {
                u32x2 v;
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    v[x] = (uint32_t)to_act_bits<DT>(o[h][i][2 * x] * inv) | (uint32_t)to_act_bits<DT>(o[h][i][2 * x + 1] * inv) << 16;
                *reinterpret_cast<u32x2_any*>(out + 16 * i) = v;
            }
        }
    }
    static constexpr int kStride = D + 4;  // of a row's partial result: m, l, two of no use, o
    static constexpr int64_t kPartial = (int64_t)kRows * kStride;
    __device__ __forceinline__ void store_partial(float* to) {
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            if (row_at(h) >= rows) continue;
            float* p = to + ((wave * HT + h) * 16 + col) * kStride;
            if (g == 0) p[0] = r[h], p[1] = l[h];
#pragma unroll
            for (int i = 0; i < NO; ++i) *reinterpret_cast<floatx4*>(p + 4 + 16 * i + 4 * g) = o[h][i];
        }
    }
};

// A block that a workgroup begins and `parts` - 1 next ones go on with (parts 0: none).
struct Record {
    int64_t b;
    int kv_head, j, parts;
};

// The cost of all blocks of one kv head of the sequences base + lane, and these.
template <class Bl>
__device__ __forceinline__ int64_t costs(const TokensArgs& a, int64_t base, int lane, Sequence& seq) {
    seq = base + lane < a.B ? Sequence(a, base + lane) : Sequence();
    const int blocks = Bl::count(a, seq.m);
    int64_t sum = 0;
    for (int j = 0; j < (blocks < 2 ? blocks : 2); ++j) sum += Bl::cost(a, seq.m, seq.n, j);
    for (uint64_t todo = __builtin_amdgcn_ballot_w64(blocks > 2); todo != 0; todo &= todo - 1) {
        const int i = __builtin_ctzll(todo);
        const int m = __builtin_amdgcn_readlane(seq.m, i), n = __builtin_amdgcn_readlane(seq.n, i);
        const int all = Bl::count(a, m);
        int64_t part = 0;
        for (int j = 2 + lane; j < all; j += 64) part += Bl::cost(a, m, n, j);
        part = read_lane(wave_scan(part), 63);
        if (lane == i) sum += part;
    }
    return sum;
}

// The items of positions [pos, end) of the list of all blocks' tiles (sequence,
// kv head, block; a block's first kHeadTiles positions are its start), at most
// kItems of them; returns the position behind the last. `per`: positions of a
// workgroup; seq, unit: the first 64 sequences and their costs.
template <class Bl>
__device__ __forceinline__ int64_t find_items(const TokensArgs& a, int lane, int64_t pos, int64_t end, int64_t per, int wg, Sequence seq,
                                              int64_t unit, Item* items, int& found) {
    found = 0;
    int64_t before = 0;
    for (int64_t base = 0; base < a.B && pos < end && found < kItems; base += 64) {
        if (a.B > 64) unit = costs<Bl>(a, base, lane, seq);
        const int64_t unit_to = wave_scan(unit);
        for (uint64_t rest = __builtin_amdgcn_ballot_w64(unit > 0 && before + a.H * unit_to > pos); rest != 0 && pos < end && found < kItems;
             rest &= rest - 1) {
            const int at = __builtin_ctzll(rest);
            Item it;
            it.b = base + at;
            it.row = read_lane(seq.row, at);
            it.m = __builtin_amdgcn_readlane(seq.m, at);
            it.n = __builtin_amdgcn_readlane(seq.n, at);
            const int64_t of_unit = read_lane(unit, at), seq_end = before + a.H * read_lane(unit_to, at);
            const int64_t seq_begin = seq_end - a.H * of_unit;
            const int blocks = Bl::count(a, it.m);
            while (pos < end && pos < seq_end && found < kItems) {
                it.kv_head = divide(pos - seq_begin, of_unit);
                int64_t begin = seq_begin + it.kv_head * of_unit;  // of the kv head, then of block j
                int j = 0;
                for (; j < blocks; j += 64) {  // the block that holds pos
                    const int64_t cost = j + lane < blocks ? Bl::cost(a, it.m, it.n, j + lane) : 0, to = wave_scan(cost);
                    const uint64_t hit = __builtin_amdgcn_ballot_w64(begin + to > pos);
                    if (hit != 0) {
                        const int i = __builtin_ctzll(hit);
                        j += i;
                        begin += read_lane(to - cost, i);
                        break;
                    }
                    begin += read_lane(to, 63);
                }
                for (; pos < end && j < blocks && found < kItems; ++j) {
                    const int count = Bl::span(a, it.m, it.n, j).count;
                    const int64_t stop_at = begin + count + kHeadTiles, stop = stop_at < end ? stop_at : end;
                    it.j = j;
                    it.from = (int)(pos - begin) - kHeadTiles;
                    it.from = it.from > 0 ? it.from : 0;
                    it.upto = (int)(stop - begin) - kHeadTiles;
                    it.whole = it.from == 0 && stop == stop_at;
                    it.parts = it.from == 0 && stop != stop_at ? divide(stop_at - 1, per) - wg + 1 : 0;
                    if (it.upto > 0 || stop == stop_at) {  // else its tiles begin in the next workgroup
                        if (threadIdx.x == 0) items[found] = it;
                        ++found;
                    }
                    pos = stop;
                    begin = stop_at;
                }
            }
        }
        before += a.H * read_lane(unit_to, 63);
    }
    return pos;
}

template <int DT, int KIND, int D, int HT>
__global__ __launch_bounds__(256, (Attend<DT, KIND, D, HT>::kPerCU)) void attention_tokens_kernel(TokensArgs a) {
    using A = Attend<DT, KIND, D, HT>;
    using Bl = Blocks<A::kRows>;
    extern __shared__ __align__(16) unsigned char smem[];
    Item* items = reinterpret_cast<Item*>(smem + A::kBytes) - kItems;
    const int lane = threadIdx.x & 63;
    const int wgs = gridDim.x;
    // Workgroups are dealt to the 8 dies in turn: neighbours in the list of
    // blocks, which read the same keys, are put on the same one.
    const int wg = blockIdx.x % 8 * (wgs / 8) + blockIdx.x / 8;

    int64_t all = 0;
    Sequence seq;
    int64_t unit = 0;
    for (int64_t base = 0; base < a.B; base += 64) {
        unit = costs<Bl>(a, base, lane, seq);
        all += read_lane(wave_scan(unit), 63);
    }
    all *= a.H;
    int64_t per = (all + wgs - 1) >> __builtin_ctz(wgs);
    if (per < kLeastTiles + kHeadTiles) per = kLeastTiles + kHeadTiles;
    int64_t pos = wg * per;
    const int64_t end = pos + per < all ? pos + per : all;
    Record record{0, 0, 0, 0};

    A w(a, smem);
    while (pos < end) {
        int found;
        __syncthreads();  // the items before these are read
        pos = same(find_items<Bl>(a, lane, pos, end, per, wg, seq, unit, items, found));
        __syncthreads();
        found = same(found);
        if (found == 0) break;
        for (int i = 0; i < found; ++i) {
            Item it = items[i];
            it = Item{same(it.b), same(it.row), same(it.m), same(it.n), same(it.kv_head), same(it.j), same(it.from), same(it.upto),
                      same(it.parts), same(it.whole)};
            Span sp = Bl::span(a, it.m, it.n, it.j);
            sp = Span{same(sp.lo), same(sp.hi), same(sp.sk), same(sp.head), same(sp.skip), same(sp.count)};
            w.run(it, sp);
            w.finish();
            if (it.whole) {
                w.store_out(it.kv_head);
            } else {
                w.store_partial(a.partials + (2 * (int64_t)wg + (it.from == 0 ? 1 : 0)) * A::kPartial);
                if (it.parts > 0) record = Record{it.b, it.kv_head, it.j, it.parts};
            }
        }
    }
    if (threadIdx.x == 0) static_cast<Record*>(a.records)[wg] = record;
}

// Joins the parts of shared blocks: blockIdx.x the workgroup that began one. The
// parts, 68 KB for 128 rows of 128, were written on other dies; bound by their loads'
// waits: 192 blocks in about 700 parts, 11.7 us with the loads of four on their way
// together, 17 one after the other; 3.9 us where there are few.
template <int DT, int KIND, int D, int HT>
__global__ __launch_bounds__(256) void attention_join_kernel(TokensArgs a) {
    using A = Attend<DT, KIND, D, HT>;
    const Record r = static_cast<const Record*>(a.records)[blockIdx.x];
    if (r.parts == 0) return;
    const Sequence s(a, r.b);
    const int64_t first = (int64_t)r.j * A::kRows, all = (int64_t)s.m * a.group;
    const int rows = (int)(all - first < A::kRows ? all - first : A::kRows);
    const float* begun = a.partials + (2 * (int64_t)blockIdx.x + 1) * A::kPartial;
    const float* next = a.partials + 2 * ((int64_t)blockIdx.x + 1) * A::kPartial;
    for (int e = blockIdx.y * 256 + threadIdx.x; e < rows * (D / 4); e += gridDim.y * 256) {
        const int row = e / (D / 4), d = e % (D / 4) * 4;
        const int64_t at = (int64_t)row * A::kStride;
        float m = begun[at], l = begun[at + 1];
        floatx4 o = *reinterpret_cast<const floatx4*>(begun + at + 4 + d);
        constexpr int kAtOnce = 4;  // parts whose loads are on their way together
        for (int p = 0; p + 1 < r.parts; p += kAtOnce) {
            float pm[kAtOnce], pl[kAtOnce], to = m;
            floatx4 po[kAtOnce];
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) {
                const bool is = p + y + 1 < r.parts;
                const float* x = next + 2 * (is ? p + y : p) * A::kPartial + at;
                pm[y] = is ? x[0] : kLowest;
                pl[y] = is ? x[1] : 0.0f;
                po[y] = *reinterpret_cast<const floatx4*>(x + 4 + d);
                if (!is) po[y] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
            }
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) to = fmaxf(to, pm[y]);
            const float u = exp2_fast(m - to);
            m = to;
            l *= u;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] *= u;
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) {
                const float v = exp2_fast(pm[y] - to);
                l += pl[y] * v;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] += po[y][i] * v;
            }
        }
        const int i = a.token_of((uint32_t)(first + row));
        const int head = r.kv_head * a.group + (int)(first + row) - i * a.group;
        const float inv = 1.0f / (l == 0.0f ? 1.0f : l);
        u32x2 y;
#pragma unroll
        for (int x = 0; x < 2; ++x)
            y[x] = (uint32_t)to_act_bits<DT>(o[2 * x] * inv) | (uint32_t)to_act_bits<DT>(o[2 * x + 1] * inv) << 16;
        *reinterpret_cast<u32x2_any*>(a.out + (s.row + i) * a.o_ts + (int64_t)head * a.o_hs + d) = y;
    }
}

struct Shape {
    int ht;
    int64_t wgs, partial;  // workgroups, floats of a partial result
};

// Blocks of 128 rows rather than 64, a tile's operands read once for two columns of
// each lane, where their sums and queries fit the registers of two workgroups a
// CU. int8 tiles, which are turned into operands once a block, gain from them at
// heads of 192 too: prompts of 2048 tokens 656 us and 890 with 64 rows; 16 bits 539 and 389.
template <int KIND>
constexpr int kMostWide = KIND == 1 ? 192 : 128;

template <int KIND, class Fn>
void by_shape(int D, int ht, Fn&& fn) {
    using std::integral_constant;
    auto with = [&](auto d) {
        if constexpr (decltype(d)::value <= kMostWide<KIND>) {
            if (ht == 2) return fn(d, integral_constant<int, 2>{});
        }
        fn(d, integral_constant<int, 1>{});
    };
    if (D == 64) with(integral_constant<int, 64>{});
    else if (D == 128) with(integral_constant<int, 128>{});
    else if (D == 192) with(integral_constant<int, 192>{});
    else with(integral_constant<int, 256>{});
}

template <int KIND>
Shape plan(const TokensArgs& a) {
    Shape s{};
    const int64_t group = a.Hq / a.H;
    // Where sequences have more than 64 rows on average. 64 of them over 2000 tokens, heads of 128, us with
    // blocks of 64 and 128: 64 rows each 108 and 112 (int8 91 and 112), 80 rows 200 and 114 (161 and 118).
    // With few sequences 64 stays ahead for longer (4 of 128 rows: 28 and 36). Of steps that mix, 60 single
    // tokens and a prompt of 900 have 64 by this rule (118 and 123), with 8 parts of 512 tokens 128 (344 and 304).
    s.ht = a.D <= kMostWide<KIND> && a.T * group > 64 * a.B ? 2 : 1;
    by_shape<KIND>(a.D, s.ht, [&](auto d, auto ht) {
        using A = Attend<0, KIND, decltype(d)::value, decltype(ht)::value>;
        s.wgs = kCUs * A::kPerCU;
        s.partial = A::kPartial;
    });
    return s;
}
Shape plan(const TokensArgs& a, int kind) { return kind == 0 ? plan<0>(a) : plan<1>(a); }

template <int DT, int KIND>
hipError_t launch(const TokensArgs& a, const Shape& s, hipStream_t stream) {
    hipError_t e = hipSuccess;
    by_shape<KIND>(a.D, s.ht, [&](auto d, auto ht) {
        constexpr int D = decltype(d)::value, HT = decltype(ht)::value;
        using A = Attend<DT, KIND, D, HT>;
        const size_t lds = A::kBytes;
        e = allow_lds<attention_tokens_kernel<DT, KIND, D, HT>>(lds);
        if (e != hipSuccess) return;
        hipLaunchKernelGGL((attention_tokens_kernel<DT, KIND, D, HT>), dim3((unsigned)s.wgs), dim3(256), lds, stream, a);
        e = hipGetLastError();
        if (e != hipSuccess) return;
        hipLaunchKernelGGL((attention_join_kernel<DT, KIND, D, HT>), dim3((unsigned)s.wgs, 8), dim3(256), 0, stream, a);
        e = hipGetLastError();
    });
    return e;
}

}  // namespace

size_t attention_tokens_workspace(const TokensArgs& a, int kind) {
    const Shape s = plan(a, kind);
    return kCounterRegionBytes + align256((size_t)s.wgs * sizeof(Record)) + (size_t)s.wgs * 2 * s.partial * 4;
}

hipError_t launch_attention_tokens(TokensArgs a, int kind, int dtype, void* workspace, hipStream_t stream) {
    const Shape s = plan(a, kind);
    a.group = a.Hq / a.H;
    a.one_by_group = std::nextafter(1.0 / a.group, 2.0);
    const int64_t most = a.width * a.P, all = ((int64_t)1 << 31) - 1;
    a.most = (int)(most < all ? most : all);
    // A position, 2^31 below 0 at the least, minus the window stays within 64 bits.
    const int64_t every = (int64_t)1 << 32;
    a.reach = a.window > 0 && a.window < every ? a.window : every;
    // Behind the counters of other calls that a caller lets share the workspace.
    unsigned char* at = static_cast<unsigned char*>(workspace) + kCounterRegionBytes;
    a.records = at;
    a.partials = reinterpret_cast<float*>(at + align256((size_t)s.wgs * sizeof(Record)));
    if (kind == 0) return dtype == 0 ? launch<0, 0>(a, s, stream) : launch<1, 0>(a, s, stream);
    return dtype == 0 ? launch<0, 1>(a, s, stream) : launch<1, 1>(a, s, stream);
}

}  // namespace w4a16
