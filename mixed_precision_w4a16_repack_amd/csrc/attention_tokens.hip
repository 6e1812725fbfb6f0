// attention_tokens.hip -- attention of several new tokens per sequence over
// the paged key/value cache (prompts, chunks of them, trees of drafted tokens):
//   s_t = scale * q . k_t,  o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),
// over the tokens t that a row sees, in one pass with a running reference m.
#include "attention_common.h"
#include "device_common.h"
#include "internal.h"
#include "kv_layout.h"

namespace w4a16 {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;       // tokens
constexpr int kHeadTiles = 6;   // a block's start and end cost about as much as this many tiles
constexpr int kLeastTiles = 8;  // a workgroup's least share: a split costs a join

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
        const int64_t first = (int64_t)j * ROWS, last = first + ROWS - 1;
        const int i0 = (int)(first / a.group), i1 = last / a.group < m ? (int)(last / a.group) : m - 1;
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

__device__ __forceinline__ uint32_t below(int64_t x) { return x <= 0 ? 0u : (x >= 32 ? ~0u : (1u << x) - 1u); }

template <int DT, int KIND, int D, int HT>
struct Attend {
    static constexpr bool kI8 = KIND == 1;
    static constexpr bool kF16P = kI8 || DT == 0;
    static constexpr int PDT = kF16P ? 0 : 1;          // operand type of both products
    static constexpr int NP = kI8 && DT == 1 ? 1 : 2;  // operands of a probability
    static constexpr int NQ = D / 32;                  // MFMAs along d
    static constexpr int NO = D / 16;
    static constexpr int kRows = 16 * HT * kWaves;
    static constexpr int kUnits = 2 * NQ + NO;         // operands of a tile, 1024 bytes each: keys, then values
    static constexpr int kStage = kUnits * 1024 + (kI8 ? 256 : 0);  // int8: then key scales and value scales
    static constexpr int kStages = 2;
    static constexpr int kLoads = (kI8 ? kUnits / 2 : kUnits) / kWaves;  // 16-byte loads a lane for a tile
    using L = KvPlace<KIND>;
    using Pr = Prob<kF16P>;
    static_assert((kI8 ? kUnits / 2 : kUnits) % kWaves == 0, "each wave loads as much of a tile");

    const TokensArgs& a;
    unsigned char* lds;
    const int lane, wave, g, col;
    u32x4 q[HT][NQ];
    float factor[HT];
    floatx4 o[HT][NO];
    float m[HT], l[HT], c[HT], f[HT];
    // Of each column: its row of the sequence's new tokens (-1: none), what it
    // sees: tokens lo .. hi - 1 and 0 .. sk - 1, and tree bits from `past` on.
    int64_t out_row[HT];
    int head[HT];
    bool valid[HT];
    int lo[HT], hi[HT];
    int64_t past;
    int full_lo, full_hi;  // tiles in [full_lo, full_hi) are seen whole by every column of the wave
    u32x4 stage[kLoads];
    float stage_scale;

    __device__ __forceinline__ Attend(const TokensArgs& args, unsigned char* smem)
        : a(args), lds(smem), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), g(lane >> 4), col(lane & 15) {}

    __device__ __forceinline__ void begin(const Sequence& s, int kv_head, int j) {
        past = (int64_t)s.n - s.m;
        int least_hi = 0x7FFFFFFF, most_lo = 0;
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            const int64_t r = (int64_t)j * kRows + (wave * HT + h) * 16 + col;
            const int i = (int)(r / a.group);
            valid[h] = i < s.m;
            head[h] = kv_head * a.group + (int)(r - (int64_t)i * a.group);
            out_row[h] = s.row + i;
            lo[h] = 0;
            hi[h] = 0x7FFFFFFF;  // columns without a row do not count
            if (valid[h]) {
                int64_t at = past + i, end = at + 1;
                if (a.tree) {
                    int depth = 0;
                    for (int w = 0; w < a.tree_words; ++w) depth += __builtin_popcountll(a.tree[out_row[h] * a.tree_ld + w]);
                    at = past + depth - 1;
                    end = depth > 0 ? past : 0;  // past tokens; the tree's by their bits
                }
                hi[h] = end > 0 ? (int)end : 0;
                lo[h] = at + 1 > a.reach ? (int)(at + 1 - a.reach) : 0;
            }
            least_hi = hi[h] < least_hi ? hi[h] : least_hi;
            most_lo = lo[h] > most_lo ? lo[h] : most_lo;
            const uint16_t* p = a.q + out_row[h] * a.q_ts + (int64_t)head[h] * a.q_hs + 8 * g;
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                q[h][x] = u32x4{0u, 0u, 0u, 0u};
                if (valid[h]) q[h][x] = *reinterpret_cast<const u32x4_any*>(p + 32 * x);
            }
            m[h] = kLowest;
            c[h] = kLowest;
            l[h] = 0.0f;
            f[h] = 1.0f;
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

    // bf16 queries over int8: moved by a power of two to the top of fp16's range.
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
                factor[h] = __builtin_ldexpf(factor[h], -up);
            }
        }
    }

    // This wave's part of a tile, to registers and from there to a stage in LDS.
    __device__ __forceinline__ void fetch_tile(const unsigned char* rec, int sub) {
        constexpr int kKeyLoads = (kI8 ? NQ : 2 * NQ);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int unit = wave * kLoads + i;
            const unsigned char* p = unit < kKeyLoads ? rec + (int64_t)sub * kKeyLoads * 1024 + unit * 1024
                                                      : rec + L::keys_bytes(D, a.P) + (int64_t)sub * kKeyLoads * 1024 + (unit - kKeyLoads) * 1024;
            stage[i] = *(reinterpret_cast<const u32x4*>(p) + lane);
        }
        if constexpr (kI8) {
            if (wave == 0) stage_scale = reinterpret_cast<const float*>(rec + 2 * L::keys_bytes(D, a.P))[sub * kTile + (lane & 31) + (lane < 32 ? 0 : a.P)];
        }
    }
    __device__ __forceinline__ void store_tile(int which) {
        u32x4* to = reinterpret_cast<u32x4*>(lds + which * kStage);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int unit = wave * kLoads + i;
            if constexpr (kI8) {
                to[(2 * unit) * 64 + lane] = codes8_to_f16(stage[i][0], stage[i][1]);
                to[(2 * unit + 1) * 64 + lane] = codes8_to_f16(stage[i][2], stage[i][3]);
            } else {
                to[unit * 64 + lane] = stage[i];
            }
        }
        if constexpr (kI8) {
            if (wave == 0) reinterpret_cast<float*>(lds + which * kStage + kUnits * 1024)[lane] = stage_scale;
        }
    }

    // Which of the tile's 32 tokens column h sees.
    __device__ __forceinline__ uint32_t visible(int h, int at, int n) const {
        const int64_t t = at;
        uint32_t seen = below(hi[h] - t) & (~below(lo[h] - t) | below((a.sinks < lo[h] ? a.sinks : lo[h]) - t));
        if (a.tree && valid[h] && at + kTile > past) {
            const int64_t first = t - past;  // the bit of the tile's first token
            const uint64_t* words = a.tree + out_row[h] * a.tree_ld;
            uint32_t bits = 0u;
            if (first < 0) {
                bits = (uint32_t)(words[0] << -first);
            } else if (first < 64 * (int64_t)a.tree_words) {
                const int w = (int)(first >> 6), by = (int)(first & 63);
                uint64_t v = words[w] >> by;
                if (by > 32 && w + 1 < a.tree_words) v |= words[w + 1] << (64 - by);
                bits = (uint32_t)v;
            }
            seen |= bits & below(n - t);
        }
        return seen;
    }

    __device__ __forceinline__ void work(int which, int at, int n) {
        const u32x4* tile = reinterpret_cast<const u32x4*>(lds + which * kStage);
        // s[h][0..3]: tokens 4g .. 4g+3 of the tile, s[h][4..7]: 16 tokens on.
        floatx4 acc[HT][2];
#pragma unroll
        for (int h = 0; h < HT; ++h)
#pragma unroll
            for (int t = 0; t < 2; ++t) acc[h][t] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const u32x4 k = tile[(t * NQ + i) * 64 + lane];
#pragma unroll
                for (int h = 0; h < HT; ++h) acc[h][t] = mfma16x16x32<PDT>(k, q[h][i], acc[h][t]);
            }
        floatx4 ks[2], vs[2];
        if constexpr (kI8) {
            const float* sc = reinterpret_cast<const float*>(tile + kUnits * 64) + 4 * g;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                ks[t] = *reinterpret_cast<const floatx4*>(sc + 16 * t);
                vs[t] = *reinterpret_cast<const floatx4*>(sc + 32 + 16 * t);
            }
        }
        const bool partial = !(at + kTile <= full_hi && (at >= full_lo || at + kTile <= a.sinks));
        float s[HT][8];
        uint32_t seen[HT];
        float peak[HT];
        bool above = false;
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            seen[h] = 0xFFu;
            if (partial) {
                const uint32_t bits = visible(h, at, n);
                seen[h] = (bits >> (4 * g) & 0xFu) | (bits >> (16 + 4 * g) & 0xFu) << 4;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[h][j] = acc[h][j / 4][j % 4] * (kI8 ? ks[j / 4][j % 4] * factor[h] : factor[h]);
                if (partial && !(seen[h] >> j & 1u)) s[h][j] = -INFINITY;
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
                    if constexpr (kI8) {
                        w[h][j] = e[h][j] * vs[j / 4][j % 4] * f[h];
                        if (partial && !(seen[h] >> j & 1u)) w[h][j] = 0.0f;  // an unseen scale may be anything
                    } else {
                        w[h][j] = e[h][j];
                    }
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
                    for (int j = 0; j < 8; ++j) {
                        const float z = exp2_fast(s[h][j] - mn) * vs[j / 4][j % 4];
                        y = fmaxf(y, partial && !(seen[h] >> j & 1u) ? 0.0f : z);
                    }
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
        u32x4 p[HT][NP];
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
        const u32x4* values = tile + 2 * NQ * 64 + lane;
        if (!kI8 && partial) {
            // 0 * NaN is NaN: values that are not finite are taken out of the
            // product, and the columns that see one become NaN in its place.
            constexpr uint32_t kInf = DT == 0 ? 0x7C00u : 0x7F80u, kOne = DT == 0 ? 0x3C00u : 0x3F80u;
            bool bad = false;
#pragma unroll
            for (int i = 0; i < NO; ++i) {
                const u32x4 v = values[64 * i];
#pragma unroll
                for (int x = 0; x < 4; ++x) bad |= (v[x] & kInf) == kInf || (v[x] >> 16 & kInf) == kInf;
            }
            if (__builtin_amdgcn_ballot_w64(bad) != 0) {
                u32x4 sees[HT];
#pragma unroll
                for (int h = 0; h < HT; ++h)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        sees[h][x] = (seen[h] >> (2 * x) & 1u ? kOne : 0u) | (seen[h] >> (2 * x + 1) & 1u ? kOne << 16 : 0u);
#pragma unroll
                for (int i = 0; i < NO; ++i) {
                    u32x4 v = values[64 * i], is{0u, 0u, 0u, 0u};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        if ((v[x] & kInf) == kInf) v[x] &= 0xFFFF0000u, is[x] |= kOne;
                        if ((v[x] >> 16 & kInf) == kInf) v[x] &= 0x0000FFFFu, is[x] |= kOne << 16;
                    }
#pragma unroll
                    for (int h = 0; h < HT; ++h) {
                        const floatx4 hits = mfma16x16x32<PDT>(is, sees[h], floatx4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                        for (int j = 0; j < NP; ++j) o[h][i] = mfma16x16x32<PDT>(v, p[h][j], o[h][i]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[h][i][r] = hits[r] > 0.0f ? NAN : o[h][i][r];
                    }
                }
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < NO; ++i) {
            const u32x4 v = values[64 * i];
#pragma unroll
            for (int j = 0; j < NP; ++j)
#pragma unroll
                for (int h = 0; h < HT; ++h) o[h][i] = mfma16x16x32<PDT>(v, p[h][j], o[h][i]);
        }
    }

    // Items [from, to) of the block's tiles, those of missing pages left out.
    __device__ __forceinline__ void run(int64_t b, int kv_head, const Span& sp, int n, int from, int to) {
        const int tiles_per_page = a.P / kTile;
        const int whole_shift = (tiles_per_page & (tiles_per_page - 1)) == 0 ? __builtin_ctz(tiles_per_page) : -1;
        int block = from;  // first item of the 64 in hand
        uint64_t todo = 0;
        int64_t place = 0;
        int sub_l = 0;
        const unsigned char* rec = nullptr;
        int sub = 0, tile = 0;
        auto next = [&]() -> bool {  // the next tile's place, if there is one
            while (todo == 0 && block < to) {
                const int item = block + lane, tile_l = sp.tile(item);
                int64_t page = -1;
                if (item < to) {
                    const int at = whole_shift >= 0 ? tile_l >> whole_shift : tile_l / tiles_per_page;
                    page = a.table[b * a.table_ld + at];
                    sub_l = tile_l - at * tiles_per_page;
                }
                const bool ok = page >= 0 && page < a.pages;
                place = ok ? (page * a.H + kv_head) * L::record_bytes(D, a.P) : 0;
                todo = __builtin_amdgcn_ballot_w64(ok);
                if (todo == 0) block += 64;
            }
            if (todo == 0) return false;
            const int i = __builtin_ctzll(todo);
            todo &= todo - 1;
            rec = a.cache + read_lane(place, i);
            sub = __builtin_amdgcn_readlane(sub_l, i);
            tile = sp.tile(block + i);
            if (todo == 0) block += 64;
            return true;
        };
        if (!next()) return;
        __syncthreads();  // the stages are free
        fetch_tile(rec, sub);
        store_tile(0);
        int at = tile * kTile, which = 0;
        bool more = next();
        __syncthreads();
        while (true) {
            if (more) fetch_tile(rec, sub);
            work(which, at, n);
            if (!more) break;
            store_tile(which ^ 1);
            at = tile * kTile;
            which ^= 1;
            more = next();
            __syncthreads();
        }
    }

    // The columns' sums, relative to m.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            l[h] = column_sum(l[h]);
            if constexpr (kI8) {
                const float back = exp2_fast(c[h] - Pr::kBias - m[h]);
#pragma unroll
                for (int i = 0; i < NO; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[h][i][r] *= back;
            }
        }
    }
    __device__ __forceinline__ void store_out() {
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            if (!valid[h]) continue;
            const float inv = 1.0f / (l[h] == 0.0f ? 1.0f : l[h]);
            uint16_t* out = a.out + out_row[h] * a.o_ts + (int64_t)head[h] * a.o_hs + 4 * g;
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
            if (!valid[h]) continue;
            float* p = to + ((wave * HT + h) * 16 + col) * kStride;
            if (g == 0) p[0] = m[h], p[1] = l[h];
#pragma unroll
            for (int i = 0; i < NO; ++i) *reinterpret_cast<floatx4*>(p + 4 + 16 * i + 4 * g) = o[h][i];
        }
    }
};

// A block that several workgroups share: begun by one, ended by `last`.
struct Record {
    int64_t b;
    int kv_head, j, last, parts;
};

template <int DT, int KIND, int D, int HT>
__global__ __launch_bounds__(256, 2) void attention_tokens_kernel(TokensArgs a) {
    using A = Attend<DT, KIND, D, HT>;
    using Bl = Blocks<A::kRows>;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63;
    const int wgs = gridDim.x;
    // Workgroups are dealt to the 8 dies in turn: neighbours in the list of
    // blocks, which read the same keys, are put on the same one.
    const int wg = wgs % 8 == 0 ? blockIdx.x % 8 * (wgs / 8) + blockIdx.x / 8 : blockIdx.x;
    Record record{0, 0, 0, 0, 0};

    // Cost of all blocks of one kv head, of the sequences base + lane.
    Sequence seq;
    auto costs = [&](int64_t base) -> int64_t {
        seq = base + lane < a.B ? Sequence(a, base + lane) : Sequence();
        const int blocks = Bl::count(a, seq.m);
        int64_t sum = 0;
        for (int j = 0; j < (blocks < 4 ? blocks : 4); ++j) sum += Bl::cost(a, seq.m, seq.n, j);
        uint64_t todo = __builtin_amdgcn_ballot_w64(blocks > 4);
        while (todo != 0) {
            const int i = __builtin_ctzll(todo);
            todo &= todo - 1;
            const int m = __builtin_amdgcn_readlane(seq.m, i), n = __builtin_amdgcn_readlane(seq.n, i);
            const int all = Bl::count(a, m);
            int64_t part = 0;
            for (int j = 4 + lane; j < all; j += 64) part += Bl::cost(a, m, n, j);
            part = read_lane(wave_scan(part), 63);
            if (lane == i) sum += part;
        }
        return sum;
    };
    int64_t unit = 0, unit_to = 0, all = 0, before = 0;
    for (int64_t base = 0; base < a.B; base += 64) {
        unit = costs(base);
        unit_to = wave_scan(unit);
        all += read_lane(unit_to, 63);
    }
    all *= a.H;
    int64_t per = (all + wgs - 1) / wgs;
    if (per < kLeastTiles + kHeadTiles) per = kLeastTiles + kHeadTiles;
    int64_t pos = wg * per;
    const int64_t end = pos + per < all ? pos + per : all;

    A w(a, smem);
    int64_t base = a.B > 64 ? -64 : 0;
    uint64_t rest = 0;  // sequences of the 64 in hand that hold pos or come behind it
    if (a.B <= 64) rest = __builtin_amdgcn_ballot_w64(unit > 0 && a.H * unit_to > pos);
    while (pos < end) {
        while (rest == 0 && base < a.B) {
            if (base >= 0) before += a.H * read_lane(unit_to, 63);
            base += 64;
            unit = costs(base);
            unit_to = wave_scan(unit);
            rest = __builtin_amdgcn_ballot_w64(unit > 0 && before + a.H * unit_to > pos);
        }
        if (rest == 0) break;
        const int at = __builtin_ctzll(rest);
        rest &= rest - 1;
        const int64_t b = base + at;
        const int64_t of_unit = read_lane(unit, at), seq_end = before + a.H * read_lane(unit_to, at), seq_begin = seq_end - a.H * of_unit;
        Sequence s;
        s.row = read_lane(seq.row, at);
        s.m = __builtin_amdgcn_readlane(seq.m, at);
        s.n = __builtin_amdgcn_readlane(seq.n, at);
        const int blocks = Bl::count(a, s.m);
        while (pos < end && pos < seq_end) {
            const int kv_head = (int)((pos - seq_begin) / of_unit);
            int64_t begin = seq_begin + kv_head * of_unit;  // of the kv head, then of block j
            int j = 0;
            for (; j < blocks; j += 64) {  // the block that holds pos
                const int64_t cost = j + lane < blocks ? Bl::cost(a, s.m, s.n, j + lane) : 0;
                const int64_t to = wave_scan(cost);
                const uint64_t hit = __builtin_amdgcn_ballot_w64(begin + to > pos);
                if (hit != 0) {
                    const int i = __builtin_ctzll(hit);
                    j += i;
                    begin += read_lane(to - cost, i);
                    break;
                }
                begin += read_lane(to, 63);
            }
            for (; pos < end && j < blocks; ++j) {
                const Span sp = Bl::span(a, s.m, s.n, j);
                const int64_t stop_at = begin + sp.count + kHeadTiles;
                const int64_t stop = stop_at < end ? stop_at : end;
                int from = (int)(pos - begin) - kHeadTiles;
                const int upto = (int)(stop - begin) - kHeadTiles;
                const bool ends = stop == stop_at;
                from = from > 0 ? from : 0;
                pos = stop;
                if (upto > 0 || ends) {  // else its tiles begin in the next workgroup
                    w.begin(s, kv_head, j);
                    w.run(b, kv_head, sp, s.n, from, upto);
                    w.finish();
                    if (from == 0 && ends) {
                        w.store_out();
                    } else {
                        w.store_partial(a.partials + (2 * (int64_t)wg + (from == 0 ? 1 : 0)) * A::kPartial);
                        if (from == 0) {
                            const int last = (int)((stop_at - 1) / per);
                            record = {b, kv_head, j, last, last - wg + 1};
                        }
                    }
                }
                begin = stop_at;
            }
        }
    }
    if (threadIdx.x == 0) static_cast<Record*>(a.records)[wg] = record;
}

// Joins the parts of shared blocks: blockIdx.x the workgroup that began one.
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
        for (int p = 0; p + 1 < r.parts; ++p) {
            const float* x = next + 2 * p * A::kPartial + at;
            const float pm = x[0], pl = x[1];
            const floatx4 po = *reinterpret_cast<const floatx4*>(x + 4 + d);
            const float to = fmaxf(m, pm), u = exp2_fast(m - to), v = exp2_fast(pm - to);
            m = to;
            l = l * u + pl * v;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = o[i] * u + po[i] * v;
        }
        const int64_t i = (first + row) / a.group;
        const int head = r.kv_head * a.group + (int)(first + row - i * a.group);
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

template <class Fn>
void by_shape(int D, int ht, Fn&& fn) {
    using std::integral_constant;
    auto with = [&](auto d) {
        if (ht == 1) fn(d, integral_constant<int, 1>{});
        else fn(d, integral_constant<int, 2>{});
    };
    if (D == 64) with(integral_constant<int, 64>{});
    else if (D == 128) with(integral_constant<int, 128>{});
    else if (D == 192) with(integral_constant<int, 192>{});
    else with(integral_constant<int, 256>{});
}

Shape plan(const TokensArgs& a, int kind) {
    Shape s{};
    const int64_t group = a.Hq / a.H;
    s.ht = a.T * group <= 64 * a.B ? 1 : 2;
    s.wgs = 2 * kCUs;
    s.partial = 64 * s.ht * (int64_t)(a.D + 4);
    return s;
}

template <int DT, int KIND>
hipError_t launch(const TokensArgs& a, const Shape& s, hipStream_t stream) {
    hipError_t e = hipSuccess;
    by_shape(a.D, s.ht, [&](auto d, auto ht) {
        constexpr int D = decltype(d)::value, HT = decltype(ht)::value;
        using A = Attend<DT, KIND, D, HT>;
        const size_t lds = (size_t)A::kStages * A::kStage;
        e = allow_lds<attention_tokens_kernel<DT, KIND, D, HT>>(lds);
        if (e != hipSuccess) return;
        hipLaunchKernelGGL((attention_tokens_kernel<DT, KIND, D, HT>), dim3((unsigned)s.wgs), dim3(256), lds, stream, a);
        e = hipGetLastError();
        if (e != hipSuccess) return;
        hipLaunchKernelGGL((attention_join_kernel<DT, KIND, D, HT>), dim3((unsigned)s.wgs, 4), dim3(256), 0, stream, a);
        e = hipGetLastError();
    });
    return e;
}

}  // namespace

size_t attention_tokens_workspace(const TokensArgs& a, int kind) {
    const Shape s = plan(a, kind);
    return align256((size_t)s.wgs * sizeof(Record)) + (size_t)s.wgs * 2 * s.partial * 4;
}

hipError_t launch_attention_tokens(TokensArgs a, int kind, int dtype, void* workspace, hipStream_t stream) {
    const Shape s = plan(a, kind);
    a.group = a.Hq / a.H;
    const int64_t most = a.width * a.P, all = ((int64_t)1 << 31) - 1;
    a.most = (int)(most < all ? most : all);
    a.reach = a.window > 0 ? a.window : (int64_t)1 << 32;
    a.records = workspace;
    a.partials = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + align256((size_t)s.wgs * sizeof(Record)));
    if (kind == 0) return dtype == 0 ? launch<0, 0>(a, s, stream) : launch<1, 0>(a, s, stream);
    return dtype == 0 ? launch<0, 1>(a, s, stream) : launch<1, 1>(a, s, stream);
}

}  // namespace w4a16
