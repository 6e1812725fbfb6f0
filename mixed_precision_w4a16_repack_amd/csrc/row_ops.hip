// row_ops.hip -- the element-wise work between a decoder layer's GEMMs, one
// pass over each row:
//   norm:  h = x (+ residual),  y = h * rsqrt(mean(h^2) + eps) * weight
//   gate:  y = silu(g) * u = g / (1 + exp(-g)) * u  of a row [g | u]
// each with y in the activation dtype, or as int8 codes with one fp32 scale
// per row: the input of the W4A8 GEMM, which a separate quantiser would have
// to read back. Statistics, products and the scale are fp32; y is rounded
// once (to 16 bits, or to a code).
//
// What bounds them: bytes for many rows (8192 x 4096 with residual 41 us for 268
// MB, 6.5 TB/s; 2048 x 14336 of the gate 28 us, 6.2 TB/s; torch's copy of as
// many bytes reaches 5.3; rows of an odd width 4.9, their 16-byte pieces
// crossing lines), the chain load - reduce - store for few (1 x 4096
// 2.3 us, 64 x 4096 to codes 3.8 us). A row is read once: it stays in registers
// up to 32768 columns.
//
// Rows need no alignment beyond their element's: 16-byte accesses are made
// on any 2-byte address (global memory takes them). The up to 7 elements of a
// row's end are stored one by one and read as part of the row's last 8.
#include "device_common.h"
#include "internal.h"

namespace w4a16 {

int64_t gate_workgroups(int64_t M, int64_t K) { return (M * ((K + 7) / 8) + 255) / 256; }

namespace {

typedef u32x4 u32x4_any __attribute__((aligned(2)));

// Eight elements of a row of K from p, n of them inside the row (1 .. 8). The
// end of a row of 8 or more is taken from its last 8 elements, so that every
// lane makes one load and none waits for another's; align8 then moves them
// to the front (the rest 0). Shorter rows are read element by element.
// The elements that align8 drops may be overwritten meanwhile: where a row is
// read a second time while its output goes over it (norm_kernel, CPT 0), they
// belong to another lane's chunk. No other element is read after its store.
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int64_t n, int64_t K) {
    if (K >= 8) return *reinterpret_cast<const u32x4_any*>(p + (n < 8 ? n - 8 : 0));
    u32x4 v{0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    return v;
}
__device__ __forceinline__ void align8(u32x4& v, int64_t n) {  // n < 8
    const int drop = 8 - (int)n;  // leading elements that belong to the chunk before
    uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
    if (drop >= 4) {
        lo = hi;
        hi = 0;
    }
    const int bits = drop % 4 * 16;
    if (bits != 0) {
        lo = lo >> bits | hi << (64 - bits);
        hi >>= bits;
    }
    v = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

__device__ __forceinline__ void store8(uint16_t* p, int64_t n, const u32x4& v) {
    if (n >= 8) {
        *reinterpret_cast<u32x4_any*>(p) = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) p[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
}

template <int DT>
__device__ __forceinline__ float elem(const u32x4& v, int e) {
    return act_to_float<DT>((uint16_t)(v[e >> 1] >> (16 * (e & 1))));
}

template <int DT>
__device__ __forceinline__ u32x4 pack8(const float* y) {
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (uint32_t)to_act_bits<DT>(y[2 * e]) | (uint32_t)to_act_bits<DT>(y[2 * e + 1]) << 16;
    return v;
}

// |y| as its bit pattern: ordered as unsigned integers with NaN above
// infinity, so a maximum over it keeps a NaN instead of dropping it.
__device__ __forceinline__ uint32_t abs_bits(float y) { return __builtin_bit_cast(uint32_t, y) & 0x7FFFFFFFu; }

// The codes of a row whose largest magnitude is amax: rint(y * (127 / amax)),
// within [-127, 127] because amax * fp32(127 / amax) rounds to 127 at most.
// `pre` lifts rows below 1e-30, whose quotient would overflow; a row of zeros
// has factor 0.
struct CodeScale {
    float pre, inv;
    __device__ __forceinline__ explicit CodeScale(float amax) {
        pre = amax < 1e-30f ? 0x1p100f : 1.0f;
        inv = amax > 0.0f ? 127.0f / (amax * pre) : 0.0f;
    }
    __device__ __forceinline__ int code(float y) const { return (int)__builtin_rintf(y * pre * inv); }
};

// Eight codes in the stored order 0,4,1,5,2,6,3,7 (the packed weight's).
__device__ __forceinline__ uint2 codes8(const float* y, const CodeScale& s) {
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int pos = e < 4 ? 2 * e : 2 * e - 7;
        out[pos >> 2] |= ((uint32_t)s.code(y[e]) & 0xFFu) << (8 * (pos & 3));
    }
    return make_uint2(out[0], out[1]);
}

// Threads of a workgroup: one row, or four of a wave each.
template <int TPR>
constexpr int kThreads = TPR < 256 ? 256 : TPR;

// Sum and maximum over the TPR threads of a row (TPR 64: one wave, no LDS).
template <int TPR>
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& amax) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        sum += __shfl_xor(sum, off);
        const uint32_t o = __shfl_xor(amax, off);
        amax = o > amax ? o : amax;
    }
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        __shared__ float s_sum[W];
        __shared__ uint32_t s_max[W];
        if ((threadIdx.x & 63) == 0) {
            s_sum[threadIdx.x >> 6] = sum;
            s_max[threadIdx.x >> 6] = amax;
        }
        __syncthreads();
        sum = 0.0f;
        amax = 0u;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            sum += s_sum[w];
            amax = s_max[w] > amax ? s_max[w] : amax;
        }
    }
}

// One row on TPR threads. CPT > 0: the row (K <= 8 * TPR * CPT) stays in
// registers between the reduction and the output, so memory is read once.
// CPT == 0: any K, the row is read twice (residual_out is written in the
// second pass only: it may be the residual or x itself).
template <int DT, int TPR, int CPT, bool OUT8>
__global__ __launch_bounds__(kThreads<TPR>) void norm_kernel(NormArgs a) {
    const int64_t m = (int64_t)blockIdx.x * (kThreads<TPR> / TPR) + threadIdx.x / TPR;
    if (TPR == 64 && m >= a.M) return;  // TPR 64 has no barrier
    const int t = threadIdx.x % TPR;
    const uint16_t* x = a.x + m * a.ldx;
    const uint16_t* r = a.residual + m * a.ldr;
    uint16_t* ro = a.residual_out + m * a.ldro;
    const int64_t chunks = (a.K + 7) / 8;
    constexpr int R = CPT > 0 ? CPT : 1;
    float h[R][8];
    u32x4 w[R], vx[R], vr[R];
    if constexpr (CPT == 0) vr[0] = u32x4{0u, 0u, 0u, 0u};
    float sum = 0.0f;
    uint32_t amax = 0u;

    auto load = [&](int64_t c, int i) {
        const int64_t n = a.K - 8 * c;
        vx[i] = load8(x + 8 * c, n, a.K);
        if (a.residual != nullptr) vr[i] = load8(r + 8 * c, n, a.K);
        w[i] = load8(a.weight + 8 * c, n, a.K);
    };
    auto sum_up = [&](int64_t c, int i) {  // h = x (+ residual)
        const int64_t n = a.K - 8 * c;
        if (n < 8 && a.K >= 8) {
            align8(vx[i], n);
            align8(w[i], n);
            align8(vr[i], n);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = elem<DT>(vx[i], e);
        if (a.residual != nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] += elem<DT>(vr[i], e);
        }
    };
    auto reduce = [&](float* hc, const u32x4& wc) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sum += hc[e] * hc[e];
            if constexpr (OUT8) {
                const uint32_t b = abs_bits(hc[e] * elem<DT>(wc, e));
                amax = b > amax ? b : amax;
            }
        }
    };
    auto finish = [&](int64_t c, float* hc, const u32x4& wc, float rs, const CodeScale& cs) {
        const int64_t n = a.K - 8 * c;
        if (a.residual_out != nullptr) store8(ro + 8 * c, n, pack8<DT>(hc));
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = (OUT8 ? hc[e] : hc[e] * rs) * elem<DT>(wc, e);
        if constexpr (OUT8) {
            *reinterpret_cast<uint2*>(a.q + m * a.ldq + 8 * c) = codes8(y, cs);
        } else {
            store8(a.y + m * a.ldy + 8 * c, n, pack8<DT>(y));
        }
    };

    if constexpr (CPT > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t c = t + (int64_t)TPR * i;
            vx[i] = vr[i] = w[i] = u32x4{0u, 0u, 0u, 0u};
            if (c < chunks) load(c, i);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t c = t + (int64_t)TPR * i;
            sum_up(c < chunks ? c : 0, i);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) reduce(h[i], w[i]);
    } else {
        for (int64_t c = t; c < chunks; c += TPR) {
            load(c, 0);
            sum_up(c, 0);
            reduce(h[0], w[0]);
        }
    }
    row_reduce<TPR>(sum, amax);
    const float rs = 1.0f / sqrtf(sum / (float)a.K + a.eps);
    // The codes do not depend on rs: it scales the row and its maximum alike.
    const float top = __builtin_bit_cast(float, amax);
    const CodeScale cs(top);
    // A row of zeros has scale 0 also where eps is 0 and rs infinite.
    if (OUT8 && t == 0) a.xs[m] = top == 0.0f ? 0.0f : top * rs / 127.0f;
    if constexpr (CPT > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t c = t + (int64_t)TPR * i;
            if (c < chunks) finish(c, h[i], w[i], rs, cs);
        }
    } else {
        for (int64_t c = t; c < chunks; c += TPR) {
            load(c, 0);
            sum_up(c, 0);
            finish(c, h[0], w[0], rs, cs);
        }
    }
}

template <int DT>
__device__ __forceinline__ void gate8(const u32x4& g, const u32x4& u, float* y) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float gf = elem<DT>(g, e);
        y[e] = gf * __builtin_amdgcn_rcpf(1.0f + __expf(-gf)) * elem<DT>(u, e);
    }
}

// 16-bit output: the chunks of 8 columns of all rows in one list, so that
// narrow rows and rows' ends leave no threads idle.
template <int DT>
__global__ __launch_bounds__(256) void gate_kernel(GateArgs a, uint32_t chunks) {  // of a row
    const int64_t first = (int64_t)blockIdx.x * 256;
    const int64_t m0 = first >> 32 == 0 ? (int64_t)((uint32_t)first / chunks) : first / chunks;
    const uint32_t at = (uint32_t)(first - m0 * chunks) + threadIdx.x;
    const uint32_t rows = at / chunks, c = at - rows * chunks;
    const int64_t m = m0 + rows;
    if (m >= a.M) return;
    const int64_t n = a.K - 8 * (int64_t)c;
    const uint16_t* x = a.x + m * a.ldx + 8 * (int64_t)c;
    u32x4 g = load8(x, n, a.K), u = load8(x + a.K, n, a.K);
    if (n < 8 && a.K >= 8) {
        align8(g, n);
        align8(u, n);
    }
    float y[8];
    gate8<DT>(g, u, y);
    store8(a.y + m * a.ldy + 8 * (int64_t)c, n, pack8<DT>(y));
}

// The same for codes, whose rounding steps are far apart: an error of the
// quotient moves a code to its neighbour with that probability, and the fast
// form is off by |g| last places (exp's argument), which is visible next to
// fp16's rounding. Here the argument is in two parts: a few last places
// (4096 x 3000 to codes 13.4 us, 12.6 with the fast form). The second part
// counts only where the first one's exp is neither 0 nor infinity: outside,
// 1 + e is 1 or infinity whatever it is, and inf * (rest <= 0) + inf, or the
// rest of an infinite argument, would be NaN.
__device__ __forceinline__ float gate_exact(float g, float u) {
    constexpr float kLog2e = 1.44269504f, kRest = 1.92596299e-8f, kLn2 = 0.693147181f;
    const float p = -g * kLog2e;
    const float rest = __builtin_fmaf(-g, kRest, __builtin_fmaf(-g, kLog2e, -p));
    float e = __builtin_amdgcn_exp2f(p);
    if (__builtin_fabsf(p) < 128.0f) e = __builtin_fmaf(e, rest * kLn2, e);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// Codes: one row on TPR threads, held in registers (CPT > 0) or computed
// twice (CPT == 0, any K).
template <int DT, int TPR, int CPT>
__global__ __launch_bounds__(kThreads<TPR>) void gate8_kernel(GateArgs a) {
    const int64_t m = (int64_t)blockIdx.x * (kThreads<TPR> / TPR) + threadIdx.x / TPR;
    if (TPR == 64 && m >= a.M) return;
    const int t = threadIdx.x % TPR;
    const uint16_t* x = a.x + m * a.ldx;
    const int64_t chunks = a.K / 8;
    constexpr int R = CPT > 0 ? CPT : 1;
    float y[R][8];
    float unused = 0.0f;
    uint32_t amax = 0u;
    auto load = [&](int64_t c, float* yc) {
        const u32x4 g = load8(x + 8 * c, 8, a.K), u = load8(x + a.K + 8 * c, 8, a.K);
#pragma unroll
        for (int e = 0; e < 8; ++e) yc[e] = gate_exact(elem<DT>(g, e), elem<DT>(u, e));
    };
    auto reduce = [&](const float* yc) {
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = abs_bits(yc[e]) > amax ? abs_bits(yc[e]) : amax;
    };
    if constexpr (CPT > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t c = t + (int64_t)TPR * i;
            if (c < chunks) {
                load(c, y[i]);
                reduce(y[i]);
            }
        }
    } else {
        for (int64_t c = t; c < chunks; c += TPR) {
            load(c, y[0]);
            reduce(y[0]);
        }
    }
    row_reduce<TPR>(unused, amax);
    const float top = __builtin_bit_cast(float, amax);
    const CodeScale cs(top);
    if (t == 0) a.xs[m] = top / 127.0f;
    if constexpr (CPT > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t c = t + (int64_t)TPR * i;
            if (c < chunks) *reinterpret_cast<uint2*>(a.q + m * a.ldq + 8 * c) = codes8(y[i], cs);
        }
    } else {
        for (int64_t c = t; c < chunks; c += TPR) {
            load(c, y[0]);
            *reinterpret_cast<uint2*>(a.q + m * a.ldq + 8 * c) = codes8(y[0], cs);
        }
    }
}

// Up to this many rows, those of 2048 .. 8192 columns are given 1024 threads
// instead of 256: there are CUs to spare, and each thread has fewer loads to
// wait for (256 x 8192 to codes 6.7 -> 5.4 us; 8192 x 4096 41.9 -> 49.8 us).
// Wider rows gain at any number (1000 x 16384 to codes 27.5 -> 23.6 us).
constexpr int64_t kFewRows = 512;

// Calls f with the threads per row and register chunks per thread of a width.
template <class F>
void by_width(int64_t M, int64_t K, F&& f) {
    using std::integral_constant;
    const int64_t c = (K + 7) / 8;
    const bool few = M <= kFewRows;
    if (c <= 64) f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (c <= 128) f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else if (c <= 256) f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (few && c <= 1024) f(integral_constant<int, 1024>{}, integral_constant<int, 1>{});
    else if (c <= 512) f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (c <= 1024) f(integral_constant<int, 256>{}, integral_constant<int, 4>{});
    else if (c <= 2048) f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
    else if (c <= 4096) f(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
    else f(integral_constant<int, 1024>{}, integral_constant<int, 0>{});
}

template <int DT>
void norm_dispatch(const NormArgs& a, hipStream_t stream) {
    by_width(a.M, a.K, [&](auto tpr, auto cpt) {
        constexpr int TPR = decltype(tpr)::value, CPT = decltype(cpt)::value, R = kThreads<TPR> / TPR;
        const dim3 grid((unsigned)((a.M + R - 1) / R)), block(kThreads<TPR>);
        if (a.q != nullptr) hipLaunchKernelGGL((norm_kernel<DT, TPR, CPT, true>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((norm_kernel<DT, TPR, CPT, false>), grid, block, 0, stream, a);
    });
}

template <int DT>
void gate_dispatch(const GateArgs& a, hipStream_t stream) {
    if (a.q == nullptr) {
        hipLaunchKernelGGL((gate_kernel<DT>), dim3((unsigned)gate_workgroups(a.M, a.K)), dim3(256), 0, stream, a,
                           (uint32_t)((a.K + 7) / 8));
        return;
    }
    by_width(a.M, a.K, [&](auto tpr, auto cpt) {
        constexpr int TPR = decltype(tpr)::value, CPT = decltype(cpt)::value, R = kThreads<TPR> / TPR;
        hipLaunchKernelGGL((gate8_kernel<DT, TPR, CPT>), dim3((unsigned)((a.M + R - 1) / R)), dim3(kThreads<TPR>), 0, stream, a);
    });
}

}  // namespace

int64_t row_threads(int64_t M, int64_t K) {
    int64_t n = 0;
    by_width(M, K, [&](auto tpr, auto) { n = decltype(tpr)::value; });
    return n;
}


hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t stream) {
    if (dtype == 0) norm_dispatch<0>(a, stream);
    else norm_dispatch<1>(a, stream);
    return hipGetLastError();
}

hipError_t launch_gate(const GateArgs& a, int dtype, hipStream_t stream) {
    if (dtype == 0) gate_dispatch<0>(a, stream);
    else gate_dispatch<1>(a, stream);
    return hipGetLastError();
}

}  // namespace w4a16
