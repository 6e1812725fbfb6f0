// kv_cache.hip -- writing keys and values to the paged cache and reading them
// back (layout in include/w4a16.h, kv_layout.h).
//
// int8: scale = max_d |x| / 127 in fp32 per token and head, code = 127 x / max
// rounded half to even, without the scale's own rounding (see Coder).
//
// Both are copies, bound by bytes and, below a few MB, by their chain of waits
// (slot, row, store: about 3 us); what differs between rows and tiles is the
// order. A key unit is 8 (int8: 2 x 8) neighbours of one token's row, so keys
// move as 16-byte pieces. A value unit holds 8 tokens of one d: values are
// turned in registers, each thread holding two neighbouring d of the tokens.
//
// rows kernel: one wave per (token, head, keys or values). tile kernel: one
// workgroup per 32 tokens (in the order given) and head, keys and values
// apart. Where their slots are a run that fills a tile, values move as whole
// units; where it starts or ends inside a tile, as aligned groups of 4 tokens;
// any other slots, element by element.
//
// 8 heads of 128, write and read, past the last-level cache: 8000 tokens in a
// row 16.8 and 17.7 us (3.8 TB/s: exactly the bytes needed, but 3 us of start
// and end), int8 15.8 and 14.4 (two of the four waves wait while the rows are
// quantised). Scattered 78 and 41 us, int8 41 and 28: a scattered token's row
// touches 48 pieces of 64 bytes for its 512, and the memory moves those whole
// (145 MB written and 175 MB read, by the counters, for 33), a write of a part
// of one being a read and a write.
#include "device_common.h"
#include "internal.h"
#include "kv_layout.h"

namespace w4a16 {
namespace {

typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The largest of magnitudes as their 16 bits, ordered as integers with NaN
// above infinity (so a NaN is kept: the row's scale is NaN), over lanes that
// are multiples of `step` apart.
__device__ __forceinline__ uint32_t larger(uint32_t x, uint32_t y) { return x > y ? x : y; }
__device__ __forceinline__ uint32_t pair_top(uint32_t w) { return larger(w & 0x7FFFu, w >> 16 & 0x7FFFu); }
__device__ __forceinline__ uint32_t lanes_top(uint32_t v, int step) {
    for (int off = step; off < 64; off *= 2) v = larger(v, __shfl_xor(v, off));
    return v;
}

// The codes of a row whose largest magnitude is top: 127 x / top rounded half
// to even, which is the code of x / (top / 127) without that scale's own
// rounding. 127 x is exact in fp32 (x has 11 bits), and a quotient of such
// numbers that is no tie differs from one by more than 2^-20 of itself, so
// the correctly rounded quotient gives the exact code. It is found from the row's rounded
// reciprocal: x * inv is off by less than two last places, the first
// correction by the exact remainder leaves less than one, the second none.
// `pre` (a power of two) keeps the remainders from fp32's ends.
struct Coder {
    float mul, top, inv;
    Coder() = default;
    __device__ __forceinline__ explicit Coder(float amax) {
        const float pre = amax < 1e-25f ? 0x1p90f : (amax > 1e25f ? 0x1p-90f : 1.0f);
        mul = 127.0f * pre;
        top = amax * pre;
        inv = amax == 0.0f ? 0.0f : 1.0f / top;
    }
    __device__ __forceinline__ uint32_t operator()(float x) const {
        const float p = x * mul;
        float q = p * inv;
        q = __builtin_fmaf(__builtin_fmaf(-q, top, p), inv, q);
        q = __builtin_fmaf(__builtin_fmaf(-q, top, p), inv, q);
        return (uint32_t)(uint8_t)(int)__builtin_rintf(q);
    }
};

template <int DT>
__device__ __forceinline__ float low(uint32_t w) { return act_to_float<DT>((uint16_t)w); }
template <int DT>
__device__ __forceinline__ float high(uint32_t w) { return act_to_float<DT>((uint16_t)(w >> 16)); }

struct Place {
    int64_t page;
    int t;
};
// slot = page * P + t; P is a power of two unless shift < 0.
__device__ __forceinline__ Place place_of(const KvArgs& a, int64_t slot) {
    if (a.shift >= 0) return {slot >> a.shift, (int)slot & (a.P - 1)};
    const int64_t page = (uint64_t)slot >> 32 == 0 ? (int64_t)((uint32_t)slot / (uint32_t)a.P) : slot / a.P;
    return {page, (int)(slot - page * a.P)};
}

// One wave per (token, head, keys or values), lanes over d.
template <int DT, int KIND>
__global__ __launch_bounds__(256) void kv_write_rows_kernel(KvArgs a) {
    using L = KvPlace<KIND>;
    const int lane = threadIdx.x & 63;
    const int unit = blockIdx.x * 4 + (threadIdx.x >> 6);
    const int which = unit & 1, tok = (unit >> 1) / a.H, h = (unit >> 1) - tok * a.H;
    if (tok >= a.T) return;
    const int64_t slot = a.slots[tok];
    if (slot < 0 || slot >= a.pages * a.P) return;
    const Place at = place_of(a, slot);
    const uint16_t* src = which ? a.v + tok * a.v_ts + h * a.v_hs : a.k + tok * a.k_ts + h * a.k_hs;
    unsigned char* rec = a.cache + (at.page * a.H + h) * L::record_bytes(a.D, a.P);
    if constexpr (KIND == 0) {
        for (int d = lane; d < a.D; d += 64) {
            const int64_t off = which ? L::value(at.t, d, a.D, a.P) : L::key(at.t, d, a.D);
            *reinterpret_cast<uint16_t*>(rec + off) = src[d];
        }
    } else {
        uint16_t x[kKvMaxD / 64];
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < kKvMaxD / 64; ++i) {
            x[i] = 64 * i < a.D ? src[64 * i + lane] : 0;
            top = larger(top, x[i] & 0x7FFFu);
        }
        const float amax = act_to_float<DT>((uint16_t)lanes_top(top, 1)), s = amax / 127.0f;
        const Coder code(amax);
#pragma unroll
        for (int i = 0; i < kKvMaxD / 64; ++i) {
            const int d = 64 * i + lane;
            if (64 * i < a.D) rec[which ? L::value(at.t, d, a.D, a.P) : L::key(at.t, d, a.D)] = (unsigned char)code(act_to_float<DT>(x[i]));
        }
        if (lane == 0) *reinterpret_cast<float*>(rec + L::scale(at.t, a.D, a.P, which)) = s;
    }
}

// The 32 tokens of a workgroup of the tile kernels, found by every wave: lane
// j holds token j's place.
struct Group {
    int n;         // tokens of the group
    bool run;      // their slots are a run inside the cache
    bool tile;     // which fills a tile
    int phase;     // the run's first slot % 4
    int64_t rec;   // byte offset of the lane's token's record, -1: nowhere
    int t;
    __device__ __forceinline__ Group(const KvArgs& a, int64_t t0, int h, int64_t record) {
        const int lane = threadIdx.x & 63;
        n = (int)(a.T - t0 < 32 ? a.T - t0 : 32);
        const int64_t s = lane < n ? a.slots[t0 + lane] : -1;
        const bool in = s >= 0 && s < a.pages * a.P;
        const Place p = place_of(a, in ? s : 0);
        rec = in ? (p.page * a.H + h) * record : -1;
        t = p.t;
        const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)s), hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(s >> 32));
        const int64_t first = (int64_t)((uint64_t)hi << 32 | lo);
        run = __builtin_amdgcn_ballot_w64(lane < n && !(in && s == first + lane)) == 0;
        tile = run && n == 32 && first % 32 == 0;
        phase = (int)(first & 3);
    }
    // Of token j (-1 outside the group), on any lane; all lanes of the wave call it.
    __device__ __forceinline__ int64_t rec_of(int j) const {
        const uint32_t lo = __shfl((int)(uint32_t)rec, j & 63), hi = __shfl((int)(uint32_t)(rec >> 32), j & 63);
        return j < 0 || j >= n ? -1 : (int64_t)((uint64_t)hi << 32 | lo);
    }
    __device__ __forceinline__ int t_of(int j) const { return __shfl(t, j & 63); }
};

// Words of tokens (2j, 2j + 1) of one d from two words (d, d + 1) of each.
__device__ __forceinline__ uint32_t lows(uint32_t x, uint32_t y) { return __builtin_amdgcn_perm(y, x, 0x05040100u); }
__device__ __forceinline__ uint32_t highs(uint32_t x, uint32_t y) { return __builtin_amdgcn_perm(y, x, 0x07060302u); }

// blockIdx.y: keys or values.
template <int DT, int KIND, int D>
__global__ __launch_bounds__(256) void kv_write_tile_kernel(KvArgs a) {
    using L = KvPlace<KIND>;
    __shared__ Coder s_code[32];  // int8: of the values
    const int64_t t0 = (int64_t)(blockIdx.x / a.H) * 32;
    const int h = blockIdx.x % a.H;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool keys = blockIdx.y == 0;
    const Group grp(a, t0, h, L::record_bytes(D, a.P));
    const uint16_t* src = keys ? a.k + t0 * a.k_ts + h * a.k_hs : a.v + t0 * a.v_ts + h * a.v_hs;
    const int64_t ts = keys ? a.k_ts : a.v_ts;

    if (KIND == 0 && keys) {
        // 16 tokens x 4 pieces of 8 d a wave and step.
        for (int i = threadIdx.x; i < 32 * (D / 8); i += 256) {
            const int j = i % 16 + i / (16 * (D / 8)) * 16, c = i / 16 % (D / 8);
            const int64_t rec = grp.rec_of(j);
            const int t = grp.t_of(j);
            if (rec >= 0)
                *reinterpret_cast<u32x4*>(a.cache + rec + L::key(t, 8 * c, D)) = *reinterpret_cast<const u32x4_any*>(src + j * ts + 8 * c);
        }
        return;
    }
    if (KIND == 1) {
        // Four lanes hold a row. Keys are written from here; of values it is the scale.
        if (wave < 2) {
            const int j = wave * 16 + lane % 16, g = lane / 16;
            const int64_t rec = grp.rec_of(j);
            const int t = grp.t_of(j);
            u32x4 x[D / 32];
            uint32_t top = 0u;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                x[i] = u32x4{0u, 0u, 0u, 0u};
                if (rec >= 0) x[i] = *reinterpret_cast<const u32x4_any*>(src + j * ts + 8 * g + 32 * i);
            }
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = larger(top, pair_top(x[i][e]));
            const float amax = act_to_float<DT>((uint16_t)lanes_top(top, 16)), s = amax / 127.0f;
            const Coder code(amax);
            if (rec >= 0) {
                if (g == 0) *reinterpret_cast<float*>(a.cache + rec + L::scale(t, D, a.P, keys ? 0 : 1)) = s;
                if (keys) {
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) {
                        u32x4 out;
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t p0 = x[2 * i + w / 2][w % 2 * 2], p1 = x[2 * i + w / 2][w % 2 * 2 + 1];
                            out[w] = code(low<DT>(p0)) | code(high<DT>(p0)) << 8 | code(low<DT>(p1)) << 16 | code(high<DT>(p1)) << 24;
                        }
                        *reinterpret_cast<u32x4*>(a.cache + rec + L::key(t, 64 * i + 8 * g, D)) = out;
                    }
                }
            }
            if (!keys && g == 0) s_code[j] = code;
        }
        if (keys) return;
        __syncthreads();
    }

    // Values.
    auto pair_at = [&](int j, int d) { return (uint32_t)*reinterpret_cast<const u32_any*>(src + j * ts + d); };
    if (grp.tile) {
        unsigned char* rec = a.cache + grp.rec_of(0);
        const int t = grp.t_of(0);
        if constexpr (KIND == 0) {
            for (int i = threadIdx.x; i < 4 * (D / 2); i += 256) {
                const int tg = i / (D / 2), d = i % (D / 2) * 2;
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = pair_at(j / 4 * 16 + 4 * tg + j % 4, d);
                u32x4 lo, hi;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    lo[j] = lows(w[2 * j], w[2 * j + 1]);
                    hi[j] = highs(w[2 * j], w[2 * j + 1]);
                }
                u32x4* out = reinterpret_cast<u32x4*>(rec + L::value(t + 4 * tg, d, D, a.P));
                out[0] = lo;
                out[1] = hi;
            }
        } else {
            for (int i = threadIdx.x; i < 4 * (D / 2); i += 256) {
                const int tg = i / (D / 2), d = i % (D / 2) * 2;
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = pair_at(j / 4 * 16 + 4 * tg + j % 4, d);
                u32x2 lo{0u, 0u}, hi{0u, 0u};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const Coder code = s_code[j / 4 * 16 + 4 * tg + j % 4];
                    lo[j / 4] |= code(low<DT>(w[j])) << (8 * (j % 4));
                    hi[j / 4] |= code(high<DT>(w[j])) << (8 * (j % 4));
                }
                unsigned char* out = rec + L::value(t + 4 * tg, d, D, a.P);
                *reinterpret_cast<u32x2*>(out) = lo;
                *reinterpret_cast<u32x2*>(out + 16) = hi;
            }
        }
        return;
    }
    // Groups of 4 tokens; of a run the aligned ones, from token -phase on.
    const int groups = grp.run ? 9 : 8, f = grp.run ? grp.phase : 0;
    for (int i = threadIdx.x; i < (groups * (D / 2) + 63) / 64 * 64; i += 256) {  // whole waves
        const int j0 = i / (D / 2) * 4 - f, d = i % (D / 2) * 2;
        int64_t rec[4];
        int t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // before any branch: every lane has to take part
            rec[j] = grp.rec_of(j0 + j);
            t[j] = grp.t_of(j0 + j);
        }
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = j0 + j >= 0 && j0 + j < grp.n ? pair_at(j0 + j, d) : 0u;
        if constexpr (KIND == 1) {  // codes in the low bytes of the two halves
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const Coder code = s_code[(j0 + j) & 31];
                w[j] = code(low<DT>(w[j])) | code(high<DT>(w[j])) << 16;
            }
        }
        if (grp.run && j0 >= 0 && j0 + 4 <= grp.n) {
            unsigned char* out = a.cache + rec[0] + L::value(t[0], d, D, a.P);
            if constexpr (KIND == 0) {
                *reinterpret_cast<u32x2*>(out) = u32x2{lows(w[0], w[1]), lows(w[2], w[3])};
                *reinterpret_cast<u32x2*>(out + 16) = u32x2{highs(w[0], w[1]), highs(w[2], w[3])};
            } else {
                const uint32_t a0 = w[0] | w[1] << 8, a1 = w[2] | w[3] << 8;
                *reinterpret_cast<uint32_t*>(out) = lows(a0, a1);
                *reinterpret_cast<uint32_t*>(out + 16) = highs(a0, a1);
            }
            continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (rec[j] < 0) continue;
            unsigned char* out = a.cache + rec[j] + L::value(t[j], d, D, a.P);
            if constexpr (KIND == 0) {
                *reinterpret_cast<uint16_t*>(out) = (uint16_t)w[j];
                *reinterpret_cast<uint16_t*>(out + 16) = (uint16_t)(w[j] >> 16);
            } else {
                out[0] = (unsigned char)w[j];
                out[16] = (unsigned char)(w[j] >> 16);
            }
        }
    }
}

// blockIdx.y: keys or values.
template <int DT, int KIND, int D>
__global__ __launch_bounds__(256) void kv_read_tile_kernel(KvArgs a) {
    using L = KvPlace<KIND>;
    const int64_t t0 = (int64_t)(blockIdx.x / a.H) * 32;
    const int h = blockIdx.x % a.H;
    const bool keys = blockIdx.y == 0;
    const Group grp(a, t0, h, L::record_bytes(D, a.P));
    uint16_t* dst = keys ? a.k_out + t0 * a.k_ts + h * a.k_hs : a.v_out + t0 * a.v_ts + h * a.v_hs;
    const int64_t ts = keys ? a.k_ts : a.v_ts;
    // Two values from codes (signed bytes) and their scale.
    auto two = [](uint32_t c0, uint32_t c1, float s) {
        return (uint32_t)to_act_bits<DT>((float)(int8_t)c0 * s) | (uint32_t)to_act_bits<DT>((float)(int8_t)c1 * s) << 16;
    };

    if (keys) {
        // 16 tokens x 4 units a wave and step.
        constexpr int kPieces = KIND == 0 ? D / 8 : D / 16;
        for (int i = threadIdx.x; i < 32 * kPieces; i += 256) {
            const int j = i % 16 + i / (16 * kPieces) * 16, c = i / 16 % kPieces;
            const int d = KIND == 0 ? 8 * c : c / 4 * 64 + c % 4 * 8;
            const int64_t rec = grp.rec_of(j);
            const int t = grp.t_of(j);
            if (j >= grp.n) continue;
            uint16_t* out = dst + j * ts + d;
            u32x4 x{0u, 0u, 0u, 0u};
            if (rec >= 0) x = *reinterpret_cast<const u32x4*>(a.cache + rec + L::key(t, d, D));
            if constexpr (KIND == 0) {
                *reinterpret_cast<u32x4_any*>(out) = x;
            } else {
                const float s = rec >= 0 ? *reinterpret_cast<const float*>(a.cache + rec + L::scale(t, D, a.P, 0)) : 0.0f;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    u32x4 y;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t w = x[2 * half + e / 2] >> (16 * (e % 2));
                        y[e] = two(w, w >> 8, s);
                    }
                    *reinterpret_cast<u32x4_any*>(out + 32 * half) = y;
                }
            }
        }
        return;
    }

    auto put = [&](int j, int d, uint32_t w) { *reinterpret_cast<u32_any*>(dst + j * ts + d) = w; };
    if (grp.tile) {
        const unsigned char* rec = a.cache + grp.rec_of(0);
        const int t = grp.t_of(0);
        for (int i = threadIdx.x; i < 4 * (D / 2); i += 256) {
            const int tg = i / (D / 2), d = i % (D / 2) * 2;
            const unsigned char* from = rec + L::value(t + 4 * tg, d, D, a.P);
            if constexpr (KIND == 0) {
                const u32x4 lo = *reinterpret_cast<const u32x4*>(from), hi = *reinterpret_cast<const u32x4*>(from + 16);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    put(j / 4 * 16 + 4 * tg + j % 4, d, j % 2 ? highs(lo[j / 2], hi[j / 2]) : lows(lo[j / 2], hi[j / 2]));
            } else {
                const u32x2 lo = *reinterpret_cast<const u32x2*>(from), hi = *reinterpret_cast<const u32x2*>(from + 16);
                const float* sc = reinterpret_cast<const float*>(rec + L::scale(t, D, a.P, 1)) + 4 * tg;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const floatx4 s = *reinterpret_cast<const floatx4*>(sc + 16 * half);
#pragma unroll
                    for (int j = 0; j < 4; ++j) put(16 * half + 4 * tg + j, d, two(lo[half] >> (8 * j), hi[half] >> (8 * j), s[j]));
                }
            }
        }
        return;
    }
    const int groups = grp.run ? 9 : 8, f = grp.run ? grp.phase : 0;
    for (int i = threadIdx.x; i < (groups * (D / 2) + 63) / 64 * 64; i += 256) {
        const int j0 = i / (D / 2) * 4 - f, d = i % (D / 2) * 2;
        int64_t rec[4];
        int t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // before any branch: every lane has to take part
            rec[j] = grp.rec_of(j0 + j);
            t[j] = grp.t_of(j0 + j);
        }
        if (grp.run && j0 >= 0 && j0 + 4 <= grp.n) {
            const unsigned char* from = a.cache + rec[0] + L::value(t[0], d, D, a.P);
            if constexpr (KIND == 0) {
                const u32x2 lo = *reinterpret_cast<const u32x2*>(from), hi = *reinterpret_cast<const u32x2*>(from + 16);
#pragma unroll
                for (int j = 0; j < 4; ++j) put(j0 + j, d, j % 2 ? highs(lo[j / 2], hi[j / 2]) : lows(lo[j / 2], hi[j / 2]));
            } else {
                const uint32_t lo = *reinterpret_cast<const uint32_t*>(from), hi = *reinterpret_cast<const uint32_t*>(from + 16);
                const floatx4 s = *reinterpret_cast<const floatx4*>(a.cache + rec[0] + L::scale(t[0], D, a.P, 1));
#pragma unroll
                for (int j = 0; j < 4; ++j) put(j0 + j, d, two(lo >> (8 * j), hi >> (8 * j), s[j]));
            }
            continue;
        }
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = 0u;
            if (rec[j] < 0) continue;
            const unsigned char* from = a.cache + rec[j] + L::value(t[j], d, D, a.P);
            if constexpr (KIND == 0) {
                w[j] = *reinterpret_cast<const uint16_t*>(from) | (uint32_t)*reinterpret_cast<const uint16_t*>(from + 16) << 16;
            } else {
                const float s = *reinterpret_cast<const float*>(a.cache + rec[j] + L::scale(t[j], D, a.P, 1));
                w[j] = two(from[0], from[16], s);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j0 + j >= 0 && j0 + j < grp.n) put(j0 + j, d, w[j]);
    }
}

template <int DT, int KIND>
__global__ __launch_bounds__(256) void kv_read_rows_kernel(KvArgs a) {
    using L = KvPlace<KIND>;
    const int lane = threadIdx.x & 63;
    const int unit = blockIdx.x * 4 + (threadIdx.x >> 6);
    const int which = unit & 1, tok = (unit >> 1) / a.H, h = (unit >> 1) - tok * a.H;
    if (tok >= a.T) return;
    const int64_t slot = a.slots[tok];
    const bool in = slot >= 0 && slot < a.pages * a.P;
    const Place at = place_of(a, in ? slot : 0);
    uint16_t* dst = which ? a.v_out + tok * a.v_ts + h * a.v_hs : a.k_out + tok * a.k_ts + h * a.k_hs;
    const unsigned char* rec = a.cache + (at.page * a.H + h) * L::record_bytes(a.D, a.P);
    float s = 0.0f;
    if (KIND == 1 && in) s = *reinterpret_cast<const float*>(rec + L::scale(at.t, a.D, a.P, which));
    for (int d = lane; d < a.D; d += 64) {
        uint16_t bits = 0;
        if (in) {
            const int64_t off = which ? L::value(at.t, d, a.D, a.P) : L::key(at.t, d, a.D);
            if constexpr (KIND == 0) bits = *reinterpret_cast<const uint16_t*>(rec + off);
            else bits = to_act_bits<DT>((float)(int8_t)rec[off] * s);
        }
        dst[d] = bits;
    }
}

// Up to this many (token, head), a wave for each row and part: 256 scattered
// tokens of 8 heads take 4.6 and 3.7 us by rows and 9.4 by tiles (64
// workgroups), 257 of a prompt 4.2 and 3.7 us, by tiles 4.0 and 4.0; 1024
// scattered 10.1 and 8.6 us, by tiles 9.8 and 9.3, in a row 8.4 and 7.3, by
// tiles 3.9 and 4.0.
constexpr int64_t kRowsMost = 2048;

template <class Fn>
void by_head_dim(int D, Fn&& fn) {
    using std::integral_constant;
    if (D == 64) fn(integral_constant<int, 64>{});
    else if (D == 128) fn(integral_constant<int, 128>{});
    else if (D == 192) fn(integral_constant<int, 192>{});
    else fn(integral_constant<int, 256>{});
}

template <int DT, int KIND>
void launch(const KvArgs& a, bool write, hipStream_t stream) {
    const unsigned wgs = (unsigned)kv_workgroups(a.T, a.H);
    if (a.T * a.H <= kRowsMost) {
        const dim3 grid(wgs);
        if (write) hipLaunchKernelGGL((kv_write_rows_kernel<DT, KIND>), grid, dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((kv_read_rows_kernel<DT, KIND>), grid, dim3(256), 0, stream, a);
        return;
    }
    const dim3 grid(wgs, 2);
    by_head_dim(a.D, [&](auto d) {
        if (write) hipLaunchKernelGGL((kv_write_tile_kernel<DT, KIND, decltype(d)::value>), grid, dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((kv_read_tile_kernel<DT, KIND, decltype(d)::value>), grid, dim3(256), 0, stream, a);
    });
}

hipError_t run(KvArgs a, bool write, int kind, int dtype, hipStream_t stream) {
    a.shift = (a.P & (a.P - 1)) == 0 ? __builtin_ctz(a.P) : -1;
    // 16-bit values are copied as they are: one instance serves both types.
    if (kind == 0) launch<0, 0>(a, write, stream);
    else if (dtype == 0) launch<0, 1>(a, write, stream);
    else launch<1, 1>(a, write, stream);
    return hipGetLastError();
}

}  // namespace

int64_t kv_workgroups(int64_t T, int64_t H) { return T * H <= kRowsMost ? (T * H * 2 + 3) / 4 : (T + 31) / 32 * H; }

hipError_t launch_kv_write(const KvArgs& a, int kind, int dtype, hipStream_t stream) { return run(a, true, kind, dtype, stream); }

hipError_t launch_kv_read(const KvArgs& a, int kind, int dtype, hipStream_t stream) { return run(a, false, kind, dtype, stream); }

}  // namespace w4a16
