// kv_cache.hip -- writing keys and values to the paged cache and reading them
// back (layout in include/w4a16.h, kv_layout.h).
//
// int8: scale = fp32(max_d |x|) / 127 per token and head, code = x / scale
// rounded half to even.
#include "device_common.h"
#include "internal.h"
#include "kv_layout.h"

namespace w4a16 {
namespace {

// One wave per (token, head, keys or values), lanes over d.
template <int DT, int KIND>
__global__ __launch_bounds__(256) void kv_write_kernel(KvArgs a) {
    using L = KvPlace<KIND>;
    const int lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int which = (int)(unit & 1);
    const int64_t th = unit >> 1;
    const int64_t tok = th / a.H;
    const int h = (int)(th % a.H);
    if (tok >= a.T) return;
    const int64_t slot = a.slots[tok];
    if (slot < 0 || slot >= a.pages * a.P) return;
    const int64_t page = slot / a.P;
    const int t = (int)(slot % a.P);
    const uint16_t* src = (which ? a.v + tok * a.v_ts + h * a.v_hs : a.k + tok * a.k_ts + h * a.k_hs);
    unsigned char* rec = a.cache + (page * a.H + h) * L::record_bytes(a.D, a.P);
    if constexpr (KIND == 0) {
        for (int d = lane; d < a.D; d += 64) {
            const int64_t off = which ? L::value(t, d, a.D, a.P) : L::key(t, d, a.D);
            *reinterpret_cast<uint16_t*>(rec + off) = src[d];
        }
    } else {
        float amax = 0.0f;
        for (int d = lane; d < a.D; d += 64) amax = fmaxf(amax, fabsf(act_to_float<DT>(src[d])));
        for (int off = 32; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off));
        const float s = amax / 127.0f;
        for (int d = lane; d < a.D; d += 64) {
            const float c = amax > 0.0f ? __builtin_rintf(act_to_float<DT>(src[d]) / s) : 0.0f;
            const int64_t off = which ? L::value(t, d, a.D, a.P) : L::key(t, d, a.D);
            rec[off] = (unsigned char)(int8_t)(c > 127.0f ? 127.0f : (c < -127.0f ? -127.0f : c));
        }
        if (lane == 0) *reinterpret_cast<float*>(rec + L::scale(t, a.D, a.P, which)) = s;
    }
}

template <int DT, int KIND>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs a) {
    using L = KvPlace<KIND>;
    const int lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int which = (int)(unit & 1);
    const int64_t th = unit >> 1;
    const int64_t tok = th / a.H;
    const int h = (int)(th % a.H);
    if (tok >= a.T) return;
    const int64_t slot = a.slots[tok];
    const bool in = slot >= 0 && slot < a.pages * a.P;
    const int64_t page = in ? slot / a.P : 0;
    const int t = in ? (int)(slot % a.P) : 0;
    uint16_t* dst = (which ? a.v_out + tok * a.v_ts + h * a.v_hs : a.k_out + tok * a.k_ts + h * a.k_hs);
    const unsigned char* rec = a.cache + (page * a.H + h) * L::record_bytes(a.D, a.P);
    for (int d = lane; d < a.D; d += 64) {
        uint16_t bits = 0;
        if (in) {
            const int64_t off = which ? L::value(t, d, a.D, a.P) : L::key(t, d, a.D);
            if constexpr (KIND == 0) {
                bits = *reinterpret_cast<const uint16_t*>(rec + off);
            } else {
                const float s = *reinterpret_cast<const float*>(rec + L::scale(t, a.D, a.P, which));
                bits = to_act_bits<DT>((float)(int8_t)rec[off] * s);
            }
        }
        dst[d] = bits;
    }
}

}  // namespace

int64_t kv_workgroups(int64_t T, int64_t H) { return (T * H * 2 + 3) / 4; }

hipError_t launch_kv_write(const KvArgs& a, int kind, int dtype, hipStream_t stream) {
    const dim3 grid((unsigned)kv_workgroups(a.T, a.H));
    if (kind == 0) hipLaunchKernelGGL((kv_write_kernel<0, 0>), grid, dim3(256), 0, stream, a);
    else if (dtype == 0) hipLaunchKernelGGL((kv_write_kernel<0, 1>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((kv_write_kernel<1, 1>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvArgs& a, int kind, int dtype, hipStream_t stream) {
    const dim3 grid((unsigned)kv_workgroups(a.T, a.H));
    if (kind == 0) hipLaunchKernelGGL((kv_read_kernel<0, 0>), grid, dim3(256), 0, stream, a);
    else if (dtype == 0) hipLaunchKernelGGL((kv_read_kernel<0, 1>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((kv_read_kernel<1, 1>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace w4a16
