// w4a16_api.cpp -- the C ABI of libw4a16.so (declared in include/w4a16.h):
// argument validation, geometry of the packed buffer, the dispatch on M and
// error reporting. No kernel code lives here.
//
// Validation follows the eligibility rules and launcher asserts of the pages
// (`can_implement` on the "rdna_hybrid_w4a16" pages and the MI300
// "triton_w4a16.py" page: supported quant types, fp16/bf16 activations,
// group sizes {-1, 32, 64, 128, 256}, K % group_size; the launcher asserts of
// `triton_w4a16_skinny_fmt_gemm`: unit column stride, N % 8 with zero points),
// plus the N % 16 and K % 128 alignment the gfx950 layout needs. Every message
// names the rule that failed.
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "internal.h"
#include "w4a16.h"

static_assert(W4A16_NOALLOC_MAX_WORKSPACE_BYTES == w4a16::kScratchBytes, "header and library agree on the scratch");

namespace w4a16 {
namespace {

thread_local char g_err[512] = "";

w4a16_status fail(w4a16_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return st;
}

void clear_error() { g_err[0] = '\0'; }

w4a16_status hip_fail(const char* what, hipError_t e) {
    return fail(W4A16_ERR_HIP, "%s failed: %s (%d)", what, hipGetErrorString(e), (int)e);
}

bool is_pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }

// Bounds that keep every size and offset computation of the calls within
// 64-bit arithmetic: N and K (the packed sizes are products of the two) and
// row strides in elements.
constexpr int64_t kMaxDim = (int64_t)1 << 32;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

w4a16_status check_stride(const char* name, int64_t ld) {
    if (ld > kMaxStride)
        return fail(W4A16_ERR_UNSUPPORTED, "%s=%lld is too large: row strides must be at most 2^40 elements", name,
                    (long long)ld);
    return W4A16_OK;
}

int ilog2(int64_t x) {
    int l = 0;
    while ((int64_t(1) << l) < x) ++l;
    return l;
}

// Shape and type rules shared by every call that takes a weight.
w4a16_status make_geometry(int64_t N, int64_t K, int32_t group_size, int32_t qtype, Geometry* g) {
    if (N <= 0 || K <= 0) return fail(W4A16_ERR_INVALID_ARG, "N=%lld and K=%lld must be positive", (long long)N, (long long)K);
    if (N > kMaxDim || K > kMaxDim)
        return fail(W4A16_ERR_UNSUPPORTED, "N=%lld and K=%lld must be at most 2^32", (long long)N, (long long)K);
    if (qtype != W4A16_UINT4B8 && qtype != W4A16_UINT4)
        return fail(W4A16_ERR_INVALID_ARG, "qtype=%d is not a w4a16_qtype (0 uint4b8, 1 uint4)", qtype);
    if (N % 8 != 0) return fail(W4A16_ERR_UNSUPPORTED, "N=%lld must be divisible by 8", (long long)N);
    if (K % 8 != 0) return fail(W4A16_ERR_UNSUPPORTED, "K=%lld must be divisible by 8", (long long)K);
    const int64_t Ge = group_size == -1 ? K : group_size;
    const bool listed = group_size == -1 || group_size == 32 || group_size == 64 || group_size == 128 ||
                        group_size == 256 || (int64_t)group_size == K;
    if (!listed)
        return fail(W4A16_ERR_UNSUPPORTED, "group_size=%d not supported; supported: -1, 32, 64, 128, 256 or K=%lld",
                    group_size, (long long)K);
    if (K % Ge != 0)
        return fail(W4A16_ERR_UNSUPPORTED, "K=%lld must be divisible by group_size=%d", (long long)K, group_size);
    g->N = N;
    g->Np = (N + 15) / 16 * 16;
    g->K = K;
    g->Kp = (K + 127) / 128 * 128;
    g->Ge = (int32_t)Ge;
    g->Kg_ck = K / Ge;
    if (g->Kg_ck > 1 && !is_pow2(Ge))
        return fail(W4A16_ERR_UNSUPPORTED, "group_size=%d must be a power of two when K/group_size > 1", group_size);
    // The layout stores the groups of the padded K (zero scales past K / Ge).
    g->Kg = g->Kg_ck == 1 ? 1 : g->Kp / Ge;
    g->gshift = g->Kg > 1 ? ilog2(Ge) : 0;
    g->qtype = qtype;
    g->codes_bytes = (size_t)g->Np * (size_t)g->Kp / 2;
    g->scales_off = align256(g->codes_bytes);
    size_t end = g->scales_off + (size_t)g->Np * (size_t)g->Kg * 2;
    if (qtype == W4A16_UINT4) {
        g->zeros_off = align256(end);
        end = g->zeros_off + (size_t)g->Np * (size_t)g->Kg;
    } else {
        g->zeros_off = 0;
    }
    g->total_bytes = align256(end);
    return W4A16_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int32_t resolve_path(int64_t M, int32_t path, int32_t skinny_max_m) {
    const int64_t t = skinny_max_m <= 0 ? 16 : skinny_max_m;
    if (path == W4A16_PATH_SKINNY || path == W4A16_PATH_MFMA) return path;
    return M <= t ? W4A16_PATH_SKINNY : W4A16_PATH_MFMA;
}

size_t skinny_workspace(const SkinnyPlan& p) {
    return p.ksplit > 1 ? kCounterRegionBytes + p.partial_bytes : 0;
}

w4a16_status repack_impl(const int32_t* weight, const void* weight_scale, const int32_t* weight_zero_point,
                         const CheckpointLayout& lay, int64_t N, int64_t K, int32_t group_size, int32_t qtype,
                         void* packed, size_t packed_bytes, hipStream_t stream) {
    Geometry g;
    w4a16_status st = make_geometry(N, K, group_size, qtype, &g);
    if (st != W4A16_OK) return st;
    if (weight == nullptr) return fail(W4A16_ERR_INVALID_ARG, "weight_packed is NULL");
    if (weight_scale == nullptr) return fail(W4A16_ERR_INVALID_ARG, "weight_scale is NULL");
    if (packed == nullptr) return fail(W4A16_ERR_INVALID_ARG, "packed is NULL");
    if ((reinterpret_cast<uintptr_t>(weight) & 3u) || (reinterpret_cast<uintptr_t>(weight_scale) & 1u) ||
        (reinterpret_cast<uintptr_t>(weight_zero_point) & 3u))
        return fail(W4A16_ERR_INVALID_ARG, "checkpoint tensors must be aligned to their element size");
    if (reinterpret_cast<uintptr_t>(packed) & 255u) return fail(W4A16_ERR_INVALID_ARG, "packed must be 256-byte aligned");
    if (packed_bytes < g.total_bytes)
        return fail(W4A16_ERR_SIZE, "packed_bytes=%zu is smaller than the %zu bytes the layout needs", packed_bytes,
                    g.total_bytes);
    hipError_t e = launch_repack(weight, static_cast<const uint16_t*>(weight_scale),
                                 qtype == W4A16_UINT4 ? weight_zero_point : nullptr, lay, g, packed, stream);
    if (e != hipSuccess) return hip_fail("repack launch", e);
    return W4A16_OK;
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

int32_t w4a16_abi_version(void) { return W4A16_ABI_VERSION; }

const char* w4a16_last_error(void) { return g_err; }

size_t w4a16_workspace_counter_bytes(void) { return kCounterRegionBytes; }

w4a16_status w4a16_packed_size(int64_t N, int64_t K, int32_t group_size, int32_t qtype, size_t* out_bytes) {
    clear_error();
    if (out_bytes == nullptr) return fail(W4A16_ERR_INVALID_ARG, "out_bytes is NULL");
    Geometry g;
    w4a16_status st = make_geometry(N, K, group_size, qtype, &g);
    if (st != W4A16_OK) return st;
    *out_bytes = g.total_bytes;
    return W4A16_OK;
}


w4a16_status w4a16_repack(const int32_t* weight_packed, const void* weight_scale, const int32_t* weight_zero_point,
                          int64_t N, int64_t K, int32_t group_size, int32_t qtype, void* packed, size_t packed_bytes,
                          hipStream_t stream) {
    clear_error();
    return repack_impl(weight_packed, weight_scale, weight_zero_point, CheckpointLayout{}, N, K, group_size, qtype,
                       packed, packed_bytes, stream);
}

w4a16_status w4a16_repack_layout(const int32_t* weight, int32_t weight_output_dim, int32_t weight_packed_dim,
                                 const void* weight_scale, int32_t scale_output_dim, const int32_t* weight_zero_point,
                                 int32_t zero_output_dim, int64_t N, int64_t K, int32_t group_size, int32_t qtype,
                                 void* packed, size_t packed_bytes, hipStream_t stream) {
    clear_error();
    const int32_t dims[4] = {weight_output_dim, weight_packed_dim, scale_output_dim, zero_output_dim};
    const char* names[4] = {"weight_output_dim", "weight_packed_dim", "scale_output_dim", "zero_output_dim"};
    for (int i = 0; i < 4; ++i)
        if (dims[i] != 0 && dims[i] != 1) return fail(W4A16_ERR_INVALID_ARG, "%s=%d must be 0 or 1", names[i], dims[i]);
    CheckpointLayout lay;
    lay.weight_n_first = weight_output_dim == 0;
    lay.weight_k_packed = weight_packed_dim != weight_output_dim;
    lay.scale_n_first = scale_output_dim == 0;
    lay.zero_n_first = zero_output_dim == 0;
    return repack_impl(weight, weight_scale, weight_zero_point, lay, N, K, group_size, qtype, packed, packed_bytes,
                       stream);
}

w4a16_status w4a16_unpack(const void* packed, int64_t N, int64_t K, int32_t group_size, int32_t qtype,
                          uint8_t* codes, uint16_t* scale_bits, uint8_t* zeros, hipStream_t stream) {
    clear_error();
    Geometry g;
    w4a16_status st = make_geometry(N, K, group_size, qtype, &g);
    if (st != W4A16_OK) return st;
    if (packed == nullptr) return fail(W4A16_ERR_INVALID_ARG, "packed is NULL");
    if (reinterpret_cast<uintptr_t>(packed) & 255u) return fail(W4A16_ERR_INVALID_ARG, "packed must be 256-byte aligned");
    if (reinterpret_cast<uintptr_t>(scale_bits) & 1u) return fail(W4A16_ERR_INVALID_ARG, "scale_bits must be 2-byte aligned");
    hipError_t e = launch_unpack(packed, g, codes, scale_bits, zeros, stream);
    if (e != hipSuccess) return hip_fail("unpack launch", e);
    return W4A16_OK;
}

int32_t w4a16_select_path(int64_t M, int32_t path, int32_t skinny_max_m) {
    clear_error();
    if (path != W4A16_PATH_AUTO && path != W4A16_PATH_SKINNY && path != W4A16_PATH_MFMA)
        return fail(W4A16_ERR_INVALID_ARG, "path=%d is not a w4a16_path (0 auto, 1 skinny, 2 mfma)", path);
    return resolve_path(M, path, skinny_max_m);
}

w4a16_status w4a16_workspace_size(int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t path,
                                  int32_t skinny_max_m, size_t* out_bytes) {
    clear_error();
    if (out_bytes == nullptr) return fail(W4A16_ERR_INVALID_ARG, "out_bytes is NULL");
    if (M < 0) return fail(W4A16_ERR_INVALID_ARG, "M=%lld must be >= 0", (long long)M);
    if (path != W4A16_PATH_AUTO && path != W4A16_PATH_SKINNY && path != W4A16_PATH_MFMA)
        return fail(W4A16_ERR_INVALID_ARG, "path=%d is not a w4a16_path (0 auto, 1 skinny, 2 mfma)", path);
    Geometry g;
    // The workspace does not depend on qtype; uint4b8 has the simpler rules.
    w4a16_status st = make_geometry(N, K, group_size, W4A16_UINT4B8, &g);
    if (st != W4A16_OK) return st;
    *out_bytes = 0;
    if (M > 0 && resolve_path(M, path, skinny_max_m) == W4A16_PATH_MFMA) {
        *out_bytes = mfma_workspace(plan_mfma(M, g, (size_t)-1));
        return W4A16_OK;
    }
    if (M > 0 && resolve_path(M, path, skinny_max_m) == W4A16_PATH_SKINNY) {
        const SkinnyPlan p = plan_skinny(M < 16 ? M : 16, g);
        if (p.n_groups * (int64_t)sizeof(uint32_t) > (int64_t)kCounterRegionBytes)
            return fail(W4A16_ERR_UNSUPPORTED, "N=%lld needs more split-K counters than the workspace holds",
                        (long long)N);
        *out_bytes = skinny_workspace(p);
    }
    return W4A16_OK;
}

}  // extern "C"

namespace w4a16 {
namespace {

// w4a16_gemm and w4a16_gemm_noalloc. With from_scratch, the workspace is the
// library's static device scratch, fetched only once every argument has
// passed validation and the call is known to need it.
w4a16_status gemm_impl(const void* A, int64_t M, int64_t lda, const void* packed, int64_t N, int64_t K,
                       int32_t group_size, int32_t qtype, int32_t dtype, const void* bias, void* C, int64_t ldc,
                       int32_t path, int32_t skinny_max_m, void* workspace, size_t workspace_bytes,
                       bool from_scratch, hipStream_t stream) {
    Geometry g;
    w4a16_status st = make_geometry(N, K, group_size, qtype, &g);
    if (st != W4A16_OK) return st;
    if (dtype != W4A16_F16 && dtype != W4A16_BF16)
        return fail(W4A16_ERR_INVALID_ARG, "dtype=%d is not a w4a16_dtype (0 fp16, 1 bf16)", dtype);
    if (path != W4A16_PATH_AUTO && path != W4A16_PATH_SKINNY && path != W4A16_PATH_MFMA)
        return fail(W4A16_ERR_INVALID_ARG, "path=%d is not a w4a16_path (0 auto, 1 skinny, 2 mfma)", path);
    if (M < 0) return fail(W4A16_ERR_INVALID_ARG, "M=%lld must be >= 0", (long long)M);
    if (M == 0) return W4A16_OK;
    if (A == nullptr || packed == nullptr || C == nullptr)
        return fail(W4A16_ERR_INVALID_ARG, "A, packed and C must not be NULL");
    if (lda < K) return fail(W4A16_ERR_INVALID_ARG, "lda=%lld must be >= K=%lld", (long long)lda, (long long)K);
    if (ldc < N) return fail(W4A16_ERR_INVALID_ARG, "ldc=%lld must be >= N=%lld", (long long)ldc, (long long)N);
    if ((st = check_stride("lda", lda)) != W4A16_OK || (st = check_stride("ldc", ldc)) != W4A16_OK) return st;
    if (!aligned16(A) || lda % 8 != 0)
        return fail(W4A16_ERR_UNSUPPORTED, "A must be 16-byte aligned with lda %% 8 == 0 (lda=%lld)", (long long)lda);
    if (reinterpret_cast<uintptr_t>(packed) & 255u) return fail(W4A16_ERR_INVALID_ARG, "packed must be 256-byte aligned");
    if ((reinterpret_cast<uintptr_t>(C) & 1u) || (reinterpret_cast<uintptr_t>(bias) & 1u))
        return fail(W4A16_ERR_INVALID_ARG, "C and bias must be 2-byte aligned");

    const int32_t which = resolve_path(M, path, skinny_max_m);
    if (which == W4A16_PATH_MFMA) {
        // The tiled kernels address one workgroup's tile (at most 128 rows
        // of A, 16 n-tiles = 128*K bytes of codes) with 32-bit byte offsets;
        // lda >= K makes this bound cover both.
        if ((128 * lda + K) * 2 >= (int64_t)1 << 31)
            return fail(W4A16_ERR_UNSUPPORTED, "lda=%lld is too large for the tiled path: need (128*lda + K)*2 < 2^31",
                        (long long)lda);
        // Medium M splits K over workgroups as far as the workspace holds the
        // partial tiles (none given: no split); the static scratch for the
        // allocation-free entry.
        size_t cap = from_scratch ? kScratchBytes : (workspace != nullptr ? workspace_bytes : 0);
        const MfmaPlan p = plan_mfma(M, g, cap);
        const size_t need = mfma_workspace(p);
        if (need > 0 && from_scratch) {
            hipError_t e = noalloc_scratch(stream, &workspace);
            if (e != hipSuccess) return hip_fail("static scratch set-up", e);
        }
        if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u))
            return fail(W4A16_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
        hipError_t e = launch_mfma(A, M, lda, packed, g, dtype, bias, C, ldc, p, need > 0 ? workspace : nullptr,
                                   stream);
        if (e != hipSuccess) return hip_fail("mfma kernel launch", e);
        return W4A16_OK;
    }

    // The skinny kernels address the activation rows of one launch (at most
    // 16) with 32-bit byte offsets.
    const int64_t rows = M < 16 ? M : 16;
    if (((rows - 1) * lda + K) * 2 > (int64_t)INT32_MAX)
        return fail(W4A16_ERR_UNSUPPORTED, "lda=%lld is too large for the skinny path: need ((M-1)*lda + K)*2 < 2^31",
                    (long long)lda);
    const SkinnyPlan p = plan_skinny(rows, g);
    if (p.n_groups * (int64_t)sizeof(uint32_t) > (int64_t)kCounterRegionBytes)
        return fail(W4A16_ERR_UNSUPPORTED, "N=%lld needs more split-K counters than the workspace holds", (long long)N);
    const size_t need = skinny_workspace(p);
    if (need > 0 && from_scratch) {
        if (need > kScratchBytes)
            return fail(W4A16_ERR_SIZE,
                        "this call needs %zu bytes of split-K workspace, more than the %zu bytes of the static "
                        "scratch; use w4a16_gemm with a caller workspace",
                        need, kScratchBytes);
        hipError_t e = noalloc_scratch(stream, &workspace);
        if (e != hipSuccess) return hip_fail("static scratch set-up", e);
        workspace_bytes = kScratchBytes;
    }
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < need)
            return fail(W4A16_ERR_SIZE, "workspace of %zu bytes is smaller than the %zu bytes this call needs",
                        workspace == nullptr ? (size_t)0 : workspace_bytes, need);
        if (reinterpret_cast<uintptr_t>(workspace) & 255u)
            return fail(W4A16_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    }
    // M > 16 on the forced skinny path: 16-row slices, one launch each.
    const uint16_t* a16 = static_cast<const uint16_t*>(A);
    uint16_t* c16 = static_cast<uint16_t*>(C);
    for (int64_t m0 = 0; m0 < M; m0 += 16) {
        const int64_t mm = M - m0 < 16 ? M - m0 : 16;
        hipError_t e = launch_skinny(a16 + m0 * lda, mm, lda, packed, g, dtype, bias, c16 + m0 * ldc, ldc, p,
                                     need > 0 ? workspace : nullptr, stream);
        if (e != hipSuccess) return hip_fail("skinny kernel launch", e);
    }
    return W4A16_OK;
}

}  // namespace
}  // namespace w4a16

extern "C" {

w4a16_status w4a16_gemm(const void* A, int64_t M, int64_t lda, const void* packed, int64_t N, int64_t K,
                        int32_t group_size, int32_t qtype, int32_t dtype, const void* bias, void* C, int64_t ldc,
                        int32_t path, int32_t skinny_max_m, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
    clear_error();
    return gemm_impl(A, M, lda, packed, N, K, group_size, qtype, dtype, bias, C, ldc, path, skinny_max_m, workspace,
                     workspace_bytes, false, stream);
}

w4a16_status w4a16_gemm_noalloc(const void* A, int64_t M, int64_t lda, const void* packed, int64_t N, int64_t K,
                                int32_t group_size, int32_t qtype, int32_t dtype, const void* bias, void* C,
                                int64_t ldc, int32_t path, int32_t skinny_max_m, hipStream_t stream) {
    clear_error();
    return gemm_impl(A, M, lda, packed, N, K, group_size, qtype, dtype, bias, C, ldc, path, skinny_max_m, nullptr, 0,
                     true, stream);
}


w4a16_status w4a8_quantize(const void* A, int64_t M, int64_t K, int64_t lda, int32_t dtype, int8_t* qa, int64_t ldq,
                           float* xs, hipStream_t stream) {
    clear_error();
    if (M < 0) return fail(W4A16_ERR_INVALID_ARG, "M=%lld must be >= 0", (long long)M);
    if (K <= 0) return fail(W4A16_ERR_INVALID_ARG, "K=%lld must be positive", (long long)K);
    if (dtype != W4A16_F16 && dtype != W4A16_BF16)
        return fail(W4A16_ERR_INVALID_ARG, "dtype=%d is not a w4a16_dtype (0 fp16, 1 bf16)", dtype);
    if (K % 8 != 0) return fail(W4A16_ERR_UNSUPPORTED, "K=%lld must be divisible by 8", (long long)K);
    if (lda < K) return fail(W4A16_ERR_INVALID_ARG, "lda=%lld must be >= K=%lld", (long long)lda, (long long)K);
    if (ldq < K) return fail(W4A16_ERR_INVALID_ARG, "ldq=%lld must be >= K=%lld", (long long)ldq, (long long)K);
    if (K > kMaxDim) return fail(W4A16_ERR_UNSUPPORTED, "K=%lld must be at most 2^32", (long long)K);
    w4a16_status st = check_stride("lda", lda);
    if (st != W4A16_OK || (st = check_stride("ldq", ldq)) != W4A16_OK) return st;
    if (M >= ((int64_t)1 << 31)) return fail(W4A16_ERR_UNSUPPORTED, "M=%lld is too large (one workgroup per row)", (long long)M);
    if (M == 0) return W4A16_OK;
    if (A == nullptr || qa == nullptr || xs == nullptr) return fail(W4A16_ERR_INVALID_ARG, "A, qa and xs must not be NULL");
    if (!aligned16(A) || lda % 8 != 0)
        return fail(W4A16_ERR_UNSUPPORTED, "A must be 16-byte aligned with lda %% 8 == 0 (lda=%lld)", (long long)lda);
    if ((reinterpret_cast<uintptr_t>(qa) & 7u) || ldq % 8 != 0)
        return fail(W4A16_ERR_UNSUPPORTED, "qa must be 8-byte aligned with ldq %% 8 == 0 (ldq=%lld)", (long long)ldq);
    if (reinterpret_cast<uintptr_t>(xs) & 3u) return fail(W4A16_ERR_INVALID_ARG, "xs must be 4-byte aligned");
    hipError_t e = launch_a8_quant(A, M, K, lda, dtype, qa, ldq, xs, stream);
    if (e != hipSuccess) return hip_fail("quantize kernel launch", e);
    return W4A16_OK;
}

w4a16_status w4a8_workspace_size(int64_t M, int64_t N, int64_t K, int32_t group_size, size_t* out_bytes) {
    clear_error();
    if (out_bytes == nullptr) return fail(W4A16_ERR_INVALID_ARG, "out_bytes is NULL");
    if (M < 0) return fail(W4A16_ERR_INVALID_ARG, "M=%lld must be >= 0", (long long)M);
    Geometry g;
    w4a16_status st = make_geometry(N, K, group_size, W4A16_UINT4B8, &g);
    if (st != W4A16_OK) return st;
    // The larger of the two kernels' needs: the call picks the ring kernel
    // only for 16-byte aligned activation and output rows.
    const size_t reg = M > 0 ? plan_w4a8(M, g).partial_bytes : 0;
    const size_t ring = M > 0 ? plan_w4a8(M, g, true, K, true).partial_bytes : 0;
    *out_bytes = reg > ring ? reg : ring;
    return W4A16_OK;
}

w4a16_status w4a8_gemm(const int8_t* qa, const float* xs, int64_t M, int64_t ldq, const void* packed, int64_t N,
                       int64_t K, int32_t group_size, int32_t dtype, const void* bias, void* C, int64_t ldc,
                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
    clear_error();
    Geometry g;
    // The weights are symmetric (uint4b8), as the pages' W4A8 kernel requires.
    w4a16_status st = make_geometry(N, K, group_size, W4A16_UINT4B8, &g);
    if (st != W4A16_OK) return st;
    if (M < 0) return fail(W4A16_ERR_INVALID_ARG, "M=%lld must be >= 0", (long long)M);
    if (dtype != W4A16_F16 && dtype != W4A16_BF16)
        return fail(W4A16_ERR_INVALID_ARG, "dtype=%d is not a w4a16_dtype (0 fp16, 1 bf16)", dtype);
    if (ldq < K) return fail(W4A16_ERR_INVALID_ARG, "ldq=%lld must be >= K=%lld", (long long)ldq, (long long)K);
    if (ldc < N) return fail(W4A16_ERR_INVALID_ARG, "ldc=%lld must be >= N=%lld", (long long)ldc, (long long)N);
    if ((st = check_stride("ldq", ldq)) != W4A16_OK || (st = check_stride("ldc", ldc)) != W4A16_OK) return st;
    if (M == 0) return W4A16_OK;
    if (qa == nullptr || xs == nullptr || packed == nullptr || C == nullptr)
        return fail(W4A16_ERR_INVALID_ARG, "qa, xs, packed and C must not be NULL");
    if (reinterpret_cast<uintptr_t>(packed) & 255u) return fail(W4A16_ERR_INVALID_ARG, "packed must be 256-byte aligned");
    if ((reinterpret_cast<uintptr_t>(qa) & 7u) || ldq % 8 != 0)
        return fail(W4A16_ERR_UNSUPPORTED, "qa must be 8-byte aligned with ldq %% 8 == 0 (ldq=%lld)", (long long)ldq);
    if ((reinterpret_cast<uintptr_t>(xs) & 3u) || (reinterpret_cast<uintptr_t>(C) & 1u) ||
        (reinterpret_cast<uintptr_t>(bias) & 1u))
        return fail(W4A16_ERR_INVALID_ARG, "xs must be 4-byte and C, bias 2-byte aligned");
    const bool qa16 = (reinterpret_cast<uintptr_t>(qa) & 15u) == 0 && ldq % 16 == 0;
    const bool c16 = (reinterpret_cast<uintptr_t>(C) & 15u) == 0 && ldc % 8 == 0;
    const W4a8Plan p = plan_w4a8(M, g, qa16, ldq, c16);
    if (p.blocks_m > 65535 || p.ksplit > 65535)
        return fail(W4A16_ERR_UNSUPPORTED, "M=%lld is too large for one W4A8 launch", (long long)M);
    if (p.partial_bytes > 0) {
        if (workspace == nullptr || workspace_bytes < p.partial_bytes)
            return fail(W4A16_ERR_SIZE, "a workspace of %zu bytes is smaller than the %zu bytes this call needs",
                        workspace == nullptr ? (size_t)0 : workspace_bytes, p.partial_bytes);
        if (reinterpret_cast<uintptr_t>(workspace) & 3u) return fail(W4A16_ERR_INVALID_ARG, "workspace must be 4-byte aligned");
    }
    hipError_t e = launch_w4a8(qa, xs, M, ldq, packed, g, dtype, bias, C, ldc, p, workspace, stream);
    if (e != hipSuccess) return hip_fail("w4a8 kernel launch", e);
    return W4A16_OK;
}

w4a16_status w4a16_dequant(const void* packed, int64_t N, int64_t K, int32_t group_size, int32_t qtype, int32_t dtype,
                           void* dense, int64_t ldw, hipStream_t stream) {
    clear_error();
    Geometry g;
    w4a16_status st = make_geometry(N, K, group_size, qtype, &g);
    if (st != W4A16_OK) return st;
    if (dtype != W4A16_F16 && dtype != W4A16_BF16)
        return fail(W4A16_ERR_INVALID_ARG, "dtype=%d is not a w4a16_dtype (0 fp16, 1 bf16)", dtype);
    if (packed == nullptr || dense == nullptr) return fail(W4A16_ERR_INVALID_ARG, "packed and dense must not be NULL");
    if (reinterpret_cast<uintptr_t>(packed) & 255u) return fail(W4A16_ERR_INVALID_ARG, "packed must be 256-byte aligned");
    if (ldw < K) return fail(W4A16_ERR_INVALID_ARG, "ldw=%lld must be >= K=%lld", (long long)ldw, (long long)K);
    if ((st = check_stride("ldw", ldw)) != W4A16_OK) return st;
    if (!aligned16(dense) || ldw % 8 != 0)
        return fail(W4A16_ERR_UNSUPPORTED, "dense must be 16-byte aligned with ldw %% 8 == 0 (ldw=%lld)", (long long)ldw);
    hipError_t e = launch_dequant(packed, g, dtype, dense, ldw, stream);
    if (e != hipSuccess) return hip_fail("dequant kernel launch", e);
    return W4A16_OK;
}

w4a16_status w4a16_gemm_dense(const void* A, int64_t M, int64_t lda, const void* dense, int64_t N, int64_t K,
                              int64_t ldw, int32_t dtype, const void* bias, void* C, int64_t ldc, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
    clear_error();
    if (N <= 0 || K <= 0) return fail(W4A16_ERR_INVALID_ARG, "N=%lld and K=%lld must be positive", (long long)N, (long long)K);
    if (dtype != W4A16_F16 && dtype != W4A16_BF16)
        return fail(W4A16_ERR_INVALID_ARG, "dtype=%d is not a w4a16_dtype (0 fp16, 1 bf16)", dtype);
    if (M < 0) return fail(W4A16_ERR_INVALID_ARG, "M=%lld must be >= 0", (long long)M);
    if (M == 0) return W4A16_OK;
    if (A == nullptr || dense == nullptr || C == nullptr)
        return fail(W4A16_ERR_INVALID_ARG, "A, dense and C must not be NULL");
    if (lda < K) return fail(W4A16_ERR_INVALID_ARG, "lda=%lld must be >= K=%lld", (long long)lda, (long long)K);
    if (ldw < K) return fail(W4A16_ERR_INVALID_ARG, "ldw=%lld must be >= K=%lld", (long long)ldw, (long long)K);
    if (ldc < N) return fail(W4A16_ERR_INVALID_ARG, "ldc=%lld must be >= N=%lld", (long long)ldc, (long long)N);
    w4a16_status st = check_stride("lda", lda);
    if (st != W4A16_OK || (st = check_stride("ldw", ldw)) != W4A16_OK || (st = check_stride("ldc", ldc)) != W4A16_OK)
        return st;
    if ((reinterpret_cast<uintptr_t>(A) | reinterpret_cast<uintptr_t>(dense) | reinterpret_cast<uintptr_t>(C) |
         reinterpret_cast<uintptr_t>(bias)) & 1u)
        return fail(W4A16_ERR_INVALID_ARG, "A, dense, C and bias must be 2-byte aligned");
    const char* what = "";
    const int bst = dense_gemm(A, M, lda, dense, N, K, ldw, dtype, bias, C, ldc, workspace, workspace_bytes, stream, &what);
    if (bst != 0) return fail(W4A16_ERR_HIP, "%s failed: hipblasStatus %d", what, bst);
    return W4A16_OK;
}

}  // extern "C"

namespace w4a16 {
namespace {

// The threads of one launch are counted in 32 bits.
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 1;

bool aligned_to(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

w4a16_status check_dtype(int32_t dtype) {
    if (dtype != W4A16_F16 && dtype != W4A16_BF16)
        return fail(W4A16_ERR_INVALID_ARG, "dtype=%d is not a w4a16_dtype (0 fp16, 1 bf16)", dtype);
    return W4A16_OK;
}

w4a16_status check_row_stride(const char* name, int64_t ld, const char* width, int64_t least) {
    if (ld < least) return fail(W4A16_ERR_INVALID_ARG, "%s=%lld must be >= %s=%lld", name, (long long)ld, width, (long long)least);
    return check_stride(name, ld);
}

// M rows of K elements.
w4a16_status check_rows(int64_t M, int64_t K, int32_t dtype, bool out8) {
    if (M < 0) return fail(W4A16_ERR_INVALID_ARG, "M=%lld must be >= 0", (long long)M);
    if (K <= 0) return fail(W4A16_ERR_INVALID_ARG, "K=%lld must be positive", (long long)K);
    w4a16_status st = check_dtype(dtype);
    if (st != W4A16_OK) return st;
    if (K > kMaxDim) return fail(W4A16_ERR_UNSUPPORTED, "K=%lld must be at most 2^32", (long long)K);
    if (out8 && K % 8 != 0) return fail(W4A16_ERR_UNSUPPORTED, "K=%lld must be divisible by 8", (long long)K);
    if (M > kMaxThreads / row_threads(M, K))
        return fail(W4A16_ERR_UNSUPPORTED, "M=%lld rows of K=%lld are too large for one launch", (long long)M, (long long)K);
    return W4A16_OK;
}

w4a16_status check_codes(const int8_t* qa, int64_t ldq, const float* xs) {
    if (!aligned_to(qa, 8) || ldq % 8 != 0)
        return fail(W4A16_ERR_UNSUPPORTED, "qa must be 8-byte aligned with ldq %% 8 == 0 (ldq=%lld)", (long long)ldq);
    if (!aligned_to(xs, 4)) return fail(W4A16_ERR_INVALID_ARG, "xs must be 4-byte aligned");
    return W4A16_OK;
}

w4a16_status norm_impl(const void* x, int64_t M, int64_t K, int64_t ldx, int32_t dtype, const void* weight, float eps,
                       const void* residual, int64_t ldr, void* residual_out, int64_t ldro, void* y, int64_t ldy,
                       int8_t* qa, int64_t ldq, float* xs, bool out8, hipStream_t stream) {
    w4a16_status st = check_rows(M, K, dtype, out8);
    if (st != W4A16_OK || (st = check_row_stride("ldx", ldx, "K", K)) != W4A16_OK) return st;
    if (out8 ? (st = check_row_stride("ldq", ldq, "K", K)) != W4A16_OK : (st = check_row_stride("ldy", ldy, "K", K)) != W4A16_OK)
        return st;
    if (residual != nullptr && (st = check_row_stride("ldr", ldr, "K", K)) != W4A16_OK) return st;
    if (residual_out != nullptr && (st = check_row_stride("ldro", ldro, "K", K)) != W4A16_OK) return st;
    if (!(eps >= 0.0f && eps <= 3.4e38f)) return fail(W4A16_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", (double)eps);
    if (M == 0) return W4A16_OK;
    if (x == nullptr || weight == nullptr) return fail(W4A16_ERR_INVALID_ARG, "x and weight must not be NULL");
    if (out8 ? (qa == nullptr || xs == nullptr) : y == nullptr)
        return fail(W4A16_ERR_INVALID_ARG, out8 ? "qa and xs must not be NULL" : "y must not be NULL");
    if (!aligned_to(x, 2) || !aligned_to(weight, 2) || !aligned_to(residual, 2) || !aligned_to(residual_out, 2) ||
        !aligned_to(y, 2))
        return fail(W4A16_ERR_INVALID_ARG, "x, weight, residual, residual_out and y must be 2-byte aligned");
    if (out8 && (st = check_codes(qa, ldq, xs)) != W4A16_OK) return st;
    NormArgs a;
    a.x = static_cast<const uint16_t*>(x);
    a.weight = static_cast<const uint16_t*>(weight);
    a.residual = static_cast<const uint16_t*>(residual);
    a.residual_out = static_cast<uint16_t*>(residual_out);
    a.y = static_cast<uint16_t*>(y);
    a.q = out8 ? qa : nullptr;
    a.xs = xs;
    a.M = M, a.K = K, a.ldx = ldx, a.ldr = ldr, a.ldro = ldro, a.ldy = ldy, a.ldq = ldq;
    a.eps = eps;
    hipError_t e = launch_norm(a, dtype, stream);
    if (e != hipSuccess) return hip_fail("rmsnorm kernel launch", e);
    return W4A16_OK;
}

w4a16_status gate_impl(const void* x, int64_t M, int64_t K, int64_t ldx, int32_t dtype, void* y, int64_t ldy,
                       int8_t* qa, int64_t ldq, float* xs, bool out8, hipStream_t stream) {
    w4a16_status st = check_rows(M, K, dtype, out8);
    if (st != W4A16_OK || (st = check_row_stride("ldx", ldx, "2*K", 2 * K)) != W4A16_OK) return st;
    if (out8 ? (st = check_row_stride("ldq", ldq, "K", K)) != W4A16_OK : (st = check_row_stride("ldy", ldy, "K", K)) != W4A16_OK)
        return st;
    if (M == 0) return W4A16_OK;
    if (!out8 && gate_workgroups(M, K) > kMaxThreads / 256)
        return fail(W4A16_ERR_UNSUPPORTED, "M=%lld rows of K=%lld are too large for one launch", (long long)M, (long long)K);
    if (x == nullptr) return fail(W4A16_ERR_INVALID_ARG, "x must not be NULL");
    if (out8 ? (qa == nullptr || xs == nullptr) : y == nullptr)
        return fail(W4A16_ERR_INVALID_ARG, out8 ? "qa and xs must not be NULL" : "y must not be NULL");
    if (!aligned_to(x, 2) || !aligned_to(y, 2)) return fail(W4A16_ERR_INVALID_ARG, "x and y must be 2-byte aligned");
    if (out8 && (st = check_codes(qa, ldq, xs)) != W4A16_OK) return st;
    GateArgs a;
    a.x = static_cast<const uint16_t*>(x);
    a.y = static_cast<uint16_t*>(y);
    a.q = out8 ? qa : nullptr;
    a.xs = xs;
    a.M = M, a.K = K, a.ldx = ldx, a.ldy = ldy, a.ldq = ldq;
    hipError_t e = launch_gate(a, dtype, stream);
    if (e != hipSuccess) return hip_fail("silu_mul kernel launch", e);
    return W4A16_OK;
}

// Geometry rules of a paged cache; *bytes is its size.
w4a16_status check_cache(int64_t pages, int32_t kv_heads, int32_t head_dim, int32_t page_size, int32_t kind, size_t* bytes) {
    if (kind != W4A16_KV_ACT && kind != W4A16_KV_INT8)
        return fail(W4A16_ERR_INVALID_ARG, "kind=%d is not a w4a16_kv_kind (0 act dtype, 1 int8)", kind);
    if (pages < 0) return fail(W4A16_ERR_INVALID_ARG, "pages=%lld must be >= 0", (long long)pages);
    if (kv_heads <= 0) return fail(W4A16_ERR_INVALID_ARG, "kv_heads=%d must be positive", kv_heads);
    if (head_dim != 64 && head_dim != 128 && head_dim != 192 && head_dim != 256)
        return fail(W4A16_ERR_UNSUPPORTED, "head_dim=%d not supported; supported: 64, 128, 192, 256", head_dim);
    if (page_size <= 0 || page_size % 32 != 0)
        return fail(W4A16_ERR_UNSUPPORTED, "page_size=%d must be a positive multiple of 32", page_size);
    // Together these keep a cache below 2^62 bytes, and a record's offsets in 31 bits.
    if (page_size > (1 << 16) || kv_heads > (1 << 16) || pages > ((int64_t)1 << 31) - 1)
        return fail(W4A16_ERR_UNSUPPORTED, "page_size and kv_heads must be at most 2^16, pages below 2^31");
    const int64_t values = (int64_t)page_size * head_dim;
    const int64_t record = kind == W4A16_KV_ACT ? 4 * values : 2 * values + 8 * (int64_t)page_size;
    if (__builtin_mul_overflow(record * kv_heads, pages, reinterpret_cast<int64_t*>(bytes)) || (int64_t)*bytes > ((int64_t)1 << 50))
        return fail(W4A16_ERR_UNSUPPORTED, "a cache must be at most 2^50 bytes");
    return W4A16_OK;
}

w4a16_status check_cache_buffer(const void* cache, size_t cache_bytes, size_t need) {
    if (need > 0 && cache == nullptr) return fail(W4A16_ERR_INVALID_ARG, "cache must not be NULL");
    if (!aligned16(cache)) return fail(W4A16_ERR_INVALID_ARG, "cache must be 16-byte aligned");
    if (cache_bytes < need)
        return fail(W4A16_ERR_SIZE, "cache_bytes=%zu is smaller than the %zu bytes of the cache", cache_bytes, need);
    return W4A16_OK;
}

// Strides of a [rows, heads, head_dim] tensor: any in [0, 2^40], negative ones excluded.
w4a16_status check_head_strides(const char* name, int64_t rs, int64_t hs) {
    if (rs < 0 || hs < 0) return fail(W4A16_ERR_INVALID_ARG, "%s strides must be >= 0", name);
    if (rs > kMaxStride || hs > kMaxStride)
        return fail(W4A16_ERR_UNSUPPORTED, "%s strides must be at most 2^40 elements", name);
    return W4A16_OK;
}

w4a16_status kv_impl(bool write, const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs,
                     int64_t T, const int64_t* slots, const void* cache, size_t cache_bytes, int64_t pages,
                     int32_t kv_heads, int32_t head_dim, int32_t page_size, int32_t kind, int32_t dtype,
                     hipStream_t stream) {
    size_t need = 0;
    w4a16_status st = check_cache(pages, kv_heads, head_dim, page_size, kind, &need);
    if (st != W4A16_OK || (st = check_dtype(dtype)) != W4A16_OK) return st;
    if (T < 0) return fail(W4A16_ERR_INVALID_ARG, "T=%lld must be >= 0", (long long)T);
    if ((st = check_head_strides("k", k_ts, k_hs)) != W4A16_OK || (st = check_head_strides("v", v_ts, v_hs)) != W4A16_OK)
        return st;
    if (T == 0) return W4A16_OK;
    if (T > kMaxThreads / 2 || kv_workgroups(T, kv_heads) > kMaxThreads / 256)  // tokens are counted in 31 bits
        return fail(W4A16_ERR_UNSUPPORTED, "T=%lld is too large for one launch", (long long)T);
    if (k == nullptr || v == nullptr || slots == nullptr)
        return fail(W4A16_ERR_INVALID_ARG, "k, v and slots must not be NULL");
    if (!aligned_to(k, 2) || !aligned_to(v, 2)) return fail(W4A16_ERR_INVALID_ARG, "k and v must be 2-byte aligned");
    if (!aligned_to(slots, 8)) return fail(W4A16_ERR_INVALID_ARG, "slots must be 8-byte aligned");
    if ((st = check_cache_buffer(cache, cache_bytes, need)) != W4A16_OK) return st;
    KvArgs a;
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    if (!write) {
        a.k_out = const_cast<uint16_t*>(a.k);
        a.v_out = const_cast<uint16_t*>(a.v);
    }
    a.T = T, a.k_ts = k_ts, a.k_hs = k_hs, a.v_ts = v_ts, a.v_hs = v_hs;
    a.slots = slots;
    a.cache = static_cast<unsigned char*>(const_cast<void*>(cache));
    a.pages = pages, a.H = kv_heads, a.D = head_dim, a.P = page_size;
    hipError_t e = write ? launch_kv_write(a, kind, dtype, stream) : launch_kv_read(a, kind, dtype, stream);
    if (e != hipSuccess) return hip_fail(write ? "kv_write kernel launch" : "kv_read kernel launch", e);
    return W4A16_OK;
}

// Shape rules of the attention calls.
w4a16_status check_attention(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t page_size, int64_t table_width, int64_t window) {
    if (B < 0) return fail(W4A16_ERR_INVALID_ARG, "B=%lld must be >= 0", (long long)B);
    if (q_heads <= 0 || q_heads % kv_heads != 0)
        return fail(W4A16_ERR_INVALID_ARG, "q_heads=%d must be a positive multiple of kv_heads=%d", q_heads, kv_heads);
    if (table_width < 0) return fail(W4A16_ERR_INVALID_ARG, "table_width=%lld must be >= 0", (long long)table_width);
    if (window < 0) return fail(W4A16_ERR_INVALID_ARG, "window=%lld must be >= 0", (long long)window);
    if (q_heads > (1 << 20) || B > (int64_t)1 << 31 || B * q_heads >= (int64_t)1 << 31)
        return fail(W4A16_ERR_UNSUPPORTED, "B=%lld sequences of q_heads=%d are too large for one launch", (long long)B, q_heads);
    if (table_width > (((int64_t)1 << 31) + page_size - 1) / page_size)
        return fail(W4A16_ERR_UNSUPPORTED, "table_width=%lld pages hold more than 2^31 tokens", (long long)table_width);
    // Bounds the sums over sequences that the kernel packs.
    if (B > 0 && table_width > ((int64_t)1 << 43) / page_size / B)
        return fail(W4A16_ERR_UNSUPPORTED, "a table of B=%lld rows of %lld pages holds more than 2^43 tokens", (long long)B,
                    (long long)table_width);
    return W4A16_OK;
}

}  // namespace
}  // namespace w4a16

extern "C" {

w4a16_status w4a16_rmsnorm(const void* x, int64_t M, int64_t K, int64_t ldx, int32_t dtype, const void* weight,
                           float eps, const void* residual, int64_t ldr, void* residual_out, int64_t ldro, void* y,
                           int64_t ldy, hipStream_t stream) {
    clear_error();
    return norm_impl(x, M, K, ldx, dtype, weight, eps, residual, ldr, residual_out, ldro, y, ldy, nullptr, 0, nullptr,
                     false, stream);
}

w4a16_status w4a8_rmsnorm(const void* x, int64_t M, int64_t K, int64_t ldx, int32_t dtype, const void* weight,
                          float eps, const void* residual, int64_t ldr, void* residual_out, int64_t ldro, int8_t* qa,
                          int64_t ldq, float* xs, hipStream_t stream) {
    clear_error();
    return norm_impl(x, M, K, ldx, dtype, weight, eps, residual, ldr, residual_out, ldro, nullptr, 0, qa, ldq, xs, true,
                     stream);
}

w4a16_status w4a16_silu_mul(const void* x, int64_t M, int64_t K, int64_t ldx, int32_t dtype, void* y, int64_t ldy,
                            hipStream_t stream) {
    clear_error();
    return gate_impl(x, M, K, ldx, dtype, y, ldy, nullptr, 0, nullptr, false, stream);
}

w4a16_status w4a8_silu_mul(const void* x, int64_t M, int64_t K, int64_t ldx, int32_t dtype, int8_t* qa, int64_t ldq,
                           float* xs, hipStream_t stream) {
    clear_error();
    return gate_impl(x, M, K, ldx, dtype, nullptr, 0, qa, ldq, xs, true, stream);
}

w4a16_status w4a16_kv_cache_size(int64_t pages, int32_t kv_heads, int32_t head_dim, int32_t page_size, int32_t kind,
                                 size_t* out_bytes) {
    clear_error();
    if (out_bytes == nullptr) return fail(W4A16_ERR_INVALID_ARG, "out_bytes is NULL");
    size_t need = 0;
    w4a16_status st = check_cache(pages, kv_heads, head_dim, page_size, kind, &need);
    if (st == W4A16_OK) *out_bytes = need;
    return st;
}

w4a16_status w4a16_kv_write(const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs,
                            int64_t T, const int64_t* slots, void* cache, size_t cache_bytes, int64_t pages,
                            int32_t kv_heads, int32_t head_dim, int32_t page_size, int32_t kind, int32_t dtype,
                            hipStream_t stream) {
    clear_error();
    return kv_impl(true, k, k_ts, k_hs, v, v_ts, v_hs, T, slots, cache, cache_bytes, pages, kv_heads, head_dim,
                   page_size, kind, dtype, stream);
}

w4a16_status w4a16_kv_read(const int64_t* slots, int64_t T, const void* cache, size_t cache_bytes, int64_t pages,
                           int32_t kv_heads, int32_t head_dim, int32_t page_size, int32_t kind, int32_t dtype, void* k,
                           int64_t k_ts, int64_t k_hs, void* v, int64_t v_ts, int64_t v_hs, hipStream_t stream) {
    clear_error();
    return kv_impl(false, k, k_ts, k_hs, v, v_ts, v_hs, T, slots, cache, cache_bytes, pages, kv_heads, head_dim,
                   page_size, kind, dtype, stream);
}

w4a16_status w4a16_attention_workspace_size(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                            int32_t page_size, int64_t table_width, int64_t window, int32_t kind,
                                            size_t* out_bytes) {
    clear_error();
    if (out_bytes == nullptr) return fail(W4A16_ERR_INVALID_ARG, "out_bytes is NULL");
    size_t unused = 0;
    w4a16_status st = check_cache(0, kv_heads, head_dim, page_size, kind, &unused);
    if (st != W4A16_OK || (st = check_attention(B, q_heads, kv_heads, page_size, table_width, window)) != W4A16_OK) return st;
    AttentionArgs a;
    a.B = B, a.width = table_width, a.window = window;
    a.Hq = q_heads, a.H = kv_heads, a.D = head_dim, a.P = page_size;
    *out_bytes = B > 0 ? attention_workspace(a, kind) : 0;
    return W4A16_OK;
}

w4a16_status w4a16_attention(const void* q, int64_t q_bs, int64_t q_hs, int64_t B, int32_t q_heads, const void* cache,
                             size_t cache_bytes, int64_t pages, int32_t kv_heads, int32_t head_dim, int32_t page_size,
                             int32_t kind, int32_t dtype, const int32_t* table, int64_t table_width, int64_t table_ld,
                             const int32_t* lengths, int64_t window, float scale, void* out, int64_t o_bs, int64_t o_hs,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
    clear_error();
    size_t need = 0;
    w4a16_status st = check_cache(pages, kv_heads, head_dim, page_size, kind, &need);
    if (st != W4A16_OK || (st = check_dtype(dtype)) != W4A16_OK ||
        (st = check_attention(B, q_heads, kv_heads, page_size, table_width, window)) != W4A16_OK ||
        (st = check_head_strides("q", q_bs, q_hs)) != W4A16_OK || (st = check_head_strides("out", o_bs, o_hs)) != W4A16_OK)
        return st;
    if ((st = check_row_stride("table_ld", table_ld, "table_width", table_width)) != W4A16_OK) return st;
    if (!(scale >= -3.4e38f && scale <= 3.4e38f)) return fail(W4A16_ERR_INVALID_ARG, "scale=%g must be finite", (double)scale);
    if (B == 0) return W4A16_OK;
    if (q == nullptr || out == nullptr || lengths == nullptr || (table == nullptr && table_width > 0))
        return fail(W4A16_ERR_INVALID_ARG, "q, table, lengths and out must not be NULL");
    if (!aligned_to(q, 2) || !aligned_to(out, 2)) return fail(W4A16_ERR_INVALID_ARG, "q and out must be 2-byte aligned");
    if (!aligned_to(table, 4) || !aligned_to(lengths, 4))
        return fail(W4A16_ERR_INVALID_ARG, "table and lengths must be 4-byte aligned");
    if ((st = check_cache_buffer(cache, cache_bytes, need)) != W4A16_OK) return st;
    AttentionArgs a;
    a.q = static_cast<const uint16_t*>(q);
    a.out = static_cast<uint16_t*>(out);
    a.B = B, a.q_ts = q_bs, a.q_hs = q_hs, a.o_ts = o_bs, a.o_hs = o_hs;
    a.cache = static_cast<const unsigned char*>(cache);
    a.pages = pages;
    a.table = table;
    a.width = table_width, a.table_ld = table_ld;
    a.lengths = lengths;
    a.window = window;
    a.Hq = q_heads, a.H = kv_heads, a.D = head_dim, a.P = page_size;
    a.scale = scale;
    const size_t ws_need = attention_workspace(a, kind);
    if (workspace == nullptr || workspace_bytes < ws_need)
        return fail(W4A16_ERR_SIZE, "workspace of %zu bytes is smaller than the %zu bytes this call needs",
                    workspace == nullptr ? (size_t)0 : workspace_bytes, ws_need);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(W4A16_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    hipError_t e = launch_attention(a, kind, dtype, workspace, stream);
    if (e != hipSuccess) return hip_fail("attention kernel launch", e);
    return W4A16_OK;
}

}  // extern "C"
