// attention.hip -- attention of one new token per sequence over the paged
// key/value cache (layout in include/w4a16.h, kv_layout.h):
//   s_t = scale * q . k_t,  o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),
// over the tokens t a sequence sees, in one pass with a running maximum m.
#include "device_common.h"
#include "internal.h"
#include "kv_layout.h"

namespace w4a16 {
namespace {

constexpr int kMaxD = 256;

// One workgroup per (sequence, query head); a wave takes every fourth token,
// lanes over d; the four waves' results are joined in LDS.
template <int DT, int KIND>
__global__ __launch_bounds__(256) void attention_kernel(AttentionArgs a) {
    using L = KvPlace<KIND>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t b = blockIdx.x / a.Hq;
    const int hq = (int)(blockIdx.x % a.Hq);
    const int h = hq / (a.Hq / a.H);
    int64_t n = a.lengths[b];
    n = n < 0 ? 0 : (n > a.width * a.P ? a.width * a.P : n);
    const int64_t first = a.window > 0 && n > a.window ? n - a.window : 0;
    const uint16_t* q = a.q + b * a.q_ts + hq * a.q_hs;
    float qv[kMaxD / 64], o[kMaxD / 64];
    for (int i = 0; i < kMaxD / 64; ++i) {
        qv[i] = 64 * i + lane < a.D ? act_to_float<DT>(q[64 * i + lane]) : 0.0f;
        o[i] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int64_t tok = first + wave; tok < n; tok += 4) {
        const int64_t page = a.table[b * a.table_ld + tok / a.P];
        if (page < 0 || page >= a.pages) continue;
        const int t = (int)(tok % a.P);
        const unsigned char* rec = a.cache + (page * a.H + h) * L::record_bytes(a.D, a.P);
        float s = 0.0f, v[kMaxD / 64];
        for (int i = 0; i < kMaxD / 64; ++i) {
            const int d = 64 * i + lane;
            v[i] = 0.0f;
            if (d >= a.D) continue;
            if constexpr (KIND == 0) {
                s += qv[i] * act_to_float<DT>(*reinterpret_cast<const uint16_t*>(rec + L::key(t, d, a.D)));
                v[i] = act_to_float<DT>(*reinterpret_cast<const uint16_t*>(rec + L::value(t, d, a.D, a.P)));
            } else {
                s += qv[i] * (float)(int8_t)rec[L::key(t, d, a.D)];
                v[i] = (float)(int8_t)rec[L::value(t, d, a.D, a.P)];
            }
        }
        for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off);
        float vs = 1.0f;
        if constexpr (KIND == 1) {
            s *= *reinterpret_cast<const float*>(rec + L::scale(t, a.D, a.P, 0));
            vs = *reinterpret_cast<const float*>(rec + L::scale(t, a.D, a.P, 1));
        }
        s *= a.scale;
        const float mn = fmaxf(m, s);
        const float ref = mn == -INFINITY ? 0.0f : mn;
        const float alpha = expf(m - ref), p = expf(s - ref);
        l = l * alpha + p;
        for (int i = 0; i < kMaxD / 64; ++i) o[i] = o[i] * alpha + p * vs * v[i];
        m = mn;
    }
    __shared__ float sm[4], sl[4], so[4][kMaxD];
    if (lane == 0) {
        sm[wave] = m;
        sl[wave] = l;
    }
    for (int i = 0; i < kMaxD / 64; ++i) so[wave][64 * i + lane] = o[i];
    __syncthreads();
    const float mm = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    const float ref = mm == -INFINITY ? 0.0f : mm;
    float total = 0.0f, acc = 0.0f;
    const int d = threadIdx.x;
    for (int w = 0; w < 4; ++w) {
        const float f = expf(sm[w] - ref);
        total += f * sl[w];
        acc += f * so[w][d];
    }
    if (d < a.D) a.out[b * a.o_ts + hq * a.o_hs + d] = to_act_bits<DT>(acc / (total == 0.0f ? 1.0f : total));
}

}  // namespace

hipError_t launch_attention(const AttentionArgs& a, int kind, int dtype, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * a.Hq));
    if (kind == 0 && dtype == 0) hipLaunchKernelGGL((attention_kernel<0, 0>), grid, dim3(256), 0, stream, a);
    else if (kind == 0) hipLaunchKernelGGL((attention_kernel<1, 0>), grid, dim3(256), 0, stream, a);
    else if (dtype == 0) hipLaunchKernelGGL((attention_kernel<0, 1>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((attention_kernel<1, 1>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace w4a16
