// C ABI of the BitLinear library: argument validation, device check and
// dispatch to the kernels. No allocation, no synchronisation; every call only
// enqueues work on the caller's stream. The contract of each entry point is
// documented in include/bitlinear.h.
#include "../../include/bitlinear.h"

#include <atomic>
#include <cmath>
#include <cstring>

#include "activation.hpp"
#include "bl_internal.hpp"

// Digest of the sources this library was built from, set by the build script.
#ifndef BL_SOURCE_HASH
#define BL_SOURCE_HASH "unknown"
#endif

namespace {

constexpr int64_t kMaxK = 2147483647LL / 127;  // 127 * K must fit in INT32
constexpr int kMaxDevices = 64;
// Backward products: every dimension below 2^24 keeps tile counts and the
// products of two dimensions far inside 64-bit indexing.
constexpr int64_t kMaxDim = 1LL << 24;

// Per-device result of the architecture check: 0 unknown, 1 gfx950, 2 other.
std::atomic<int> g_arch[kMaxDevices];

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool valid_dtype(int d) { return d == BL_F32 || d == BL_BF16; }
bool valid_layout(int l) { return l == BL_PACK_2BIT || l == BL_PACK_BASE3 || l == BL_PACK_1BIT; }
static_assert(BL_PACK_2BIT == bl::kLayout2Bit && BL_PACK_BASE3 == bl::kLayoutBase3 &&
                  BL_PACK_1BIT == bl::kLayout1Bit,
              "layout numbering");
bool valid_scheme(int s) { return s == BL_TERNARY || s == BL_BINARY; }

bl_status device_ok() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
        (void)hipGetLastError();
        return BL_ERR_DEVICE;
    }
    int st = g_arch[dev].load(std::memory_order_relaxed);
    if (st == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
            (void)hipGetLastError();
            return BL_ERR_DEVICE;
        }
        st = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        g_arch[dev].store(st, std::memory_order_relaxed);
    }
    return st == 1 ? BL_OK : BL_ERR_DEVICE;
}

bl_status launched(hipError_t e) {
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return BL_ERR_DEVICE;
    }
    return BL_OK;
}

int64_t row_bytes(int64_t K, int layout) { return bl::row_bytes_of(layout, K); }

// Segment table of a stacked matrix: 1..kMaxSegments host row counts, each
// >= 1. Fills `gm` (bounds = running row totals) and `N` (the total).
bool make_segments(const float *gammas, const int64_t *seg_rows, int nseg, bl::GammaMap &gm,
                   int64_t &N) {
    if (!seg_rows || nseg < 1 || nseg > bl::kMaxSegments) return false;
    gm = bl::GammaMap::single(gammas);
    gm.nseg = nseg;
    N = 0;
    for (int s = 0; s < nseg; ++s) {
        if (seg_rows[s] < 1 || seg_rows[s] > 2147483647LL - N) return false;
        N += seg_rows[s];
        if (s + 1 < nseg) gm.bound[s] = N;
    }
    return true;
}

bl_status forward_impl(const int8_t *xq, const float *scale, const uint8_t *packed, int layout,
                       const float *gamma, const bl::GammaMap &gm, int64_t M, int64_t N,
                       int64_t K, void *y, int y_dtype, int32_t *acc, void *stream) {
    if (!xq || !scale || !packed || !gamma || !y) return BL_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(scale) || !aligned16(packed) || !aligned4(gamma) ||
        !aligned16(y) || (acc && !aligned16(acc)))
        return BL_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 1 || K > kMaxK) return BL_ERR_INVALID_ARG;
    if (M > 65535LL * 128 || N > 2147483647LL) return BL_ERR_INVALID_ARG;
    if (!valid_layout(layout) || !valid_dtype(y_dtype)) return BL_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return BL_OK;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (bl::skinny_handles(M, N, K, layout))
        return launched(
            bl::launch_forward_skinny(xq, scale, packed, layout, gm, M, N, K, y, y_dtype, acc, s));
    return launched(
        bl::launch_forward_gemm(xq, scale, packed, layout, gm, M, N, K, y, y_dtype, acc, s));
}

bl_status linear_impl(const void *x, int x_dtype, const uint8_t *packed, int layout,
                      const float *gamma, const bl::GammaMap &gm, int64_t M, int64_t N, int64_t K,
                      void *y, int y_dtype, int32_t *acc, void *stream) {
    if (!x || !packed || !gamma || !y) return BL_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(packed) || !aligned4(gamma) || !aligned16(y) ||
        (acc && !aligned16(acc)))
        return BL_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 1 || K > kMaxK || N > 2147483647LL) return BL_ERR_INVALID_ARG;
    if (!valid_dtype(x_dtype) || !valid_layout(layout) || !valid_dtype(y_dtype))
        return BL_ERR_INVALID_ARG;
    if (M > bl::fused_decode_max_m()) return BL_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return BL_OK;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    return launched(bl::launch_linear_decode(x, x_dtype, packed, layout, gm, M, N, K, y, y_dtype,
                                             acc, static_cast<hipStream_t>(stream)));
}

static_assert(BL_ACT_NONE == bl::kActNone && BL_ACT_GELU_TANH == bl::kActGeluTanh &&
                  BL_NORM_LAYER == bl::kNormLayer && BL_GATE_TOKEN == bl::kGateToken,
              "enum numbering");

// Operands of the extended epilogue: what must hold whatever the product.
bool valid_epilogue(const bl::EpilogueArgs &ep) {
    if (ep.act < 0 || ep.act >= bl::kActCount || !valid_dtype(ep.bias_dtype)) return false;
    if (ep.residual && !std::isfinite(ep.res_scale)) return false;
    return aligned16(ep.bias) && aligned16(ep.residual) && aligned16(ep.z);  // NULL is aligned
}

// A stack of two matrices of F rows, and what must hold of a gated epilogue's operands.
bool make_pair(const float *gammas, int64_t F, bl::GammaMap &gm) {
    const int64_t rows[2] = {F, F};
    int64_t N = 0;
    return make_segments(gammas, rows, 2, gm, N);
}
bool valid_gated(const bl::GatedArgs &ga) {
    if (ga.act < 0 || ga.act >= bl::kActCount || !valid_dtype(ga.bias_dtype)) return false;
    if ((ga.codes != nullptr) != (ga.code_scale != nullptr)) return false;
    return aligned16(ga.bias) && aligned16(ga.z) && aligned16(ga.codes) && aligned16(ga.code_scale);
}

// One norm of the block norm: kind, and parameters only with a norm.
bool valid_norm(const bl::NormSide &s) {
    if (s.kind < bl::kNormNone || s.kind > bl::kNormLayer) return false;
    if (s.kind == bl::kNormNone) return !s.weight && !s.bias;
    return std::isfinite(s.eps) && s.eps > 0.f && aligned16(s.weight) && aligned16(s.bias);
}

}  // namespace

extern "C" {

int64_t bitlinear_packed_row_bytes(int64_t K, int layout) {
    if (K < 1 || !valid_layout(layout)) return -1;
    return row_bytes(K, layout);
}

size_t bitlinear_pack_workspace_bytes(int64_t N, int64_t K) {
    if (N < 1 || K < 1 || N > INT64_MAX / K) return 0;
    return bl::pack_workspace_bytes(N * K);
}

bl_status bitlinear_pack_weights(const void *W, int w_dtype, int64_t N, int64_t K, int scheme,
                                 int layout, float eps, uint8_t *packed, float *gamma,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    if (!W || !packed || !gamma || !workspace) return BL_ERR_INVALID_ARG;
    if (!aligned16(W) || !aligned16(packed) || !aligned4(gamma) || !aligned16(workspace))
        return BL_ERR_INVALID_ARG;
    if (N < 1 || K < 1 || K > kMaxK) return BL_ERR_INVALID_ARG;
    if (N > INT64_MAX / K) return BL_ERR_INVALID_ARG;
    if (!valid_dtype(w_dtype) || !valid_layout(layout) || !valid_scheme(scheme))
        return BL_ERR_INVALID_ARG;
    if (layout == BL_PACK_1BIT && scheme != BL_BINARY) return BL_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f) return BL_ERR_INVALID_ARG;
    if (workspace_bytes < bl::pack_workspace_bytes(N * K)) return BL_ERR_INVALID_ARG;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    return launched(bl::launch_pack(W, w_dtype, N, K, scheme, layout, eps, packed, gamma,
                                    static_cast<double *>(workspace),
                                    static_cast<hipStream_t>(stream)));
}

bl_status bitlinear_pack_weights_noalloc(const void *W, int w_dtype, int64_t N, int64_t K,
                                         int scheme, int layout, float eps, uint8_t *packed,
                                         float *gamma, void *stream) {
    if (!W || !packed || !gamma) return BL_ERR_INVALID_ARG;
    if (!aligned16(W) || !aligned16(packed) || !aligned4(gamma)) return BL_ERR_INVALID_ARG;
    if (N < 1 || K < 1 || K > kMaxK) return BL_ERR_INVALID_ARG;
    if (N > INT64_MAX / K) return BL_ERR_INVALID_ARG;
    if (!valid_dtype(w_dtype) || !valid_layout(layout) || !valid_scheme(scheme))
        return BL_ERR_INVALID_ARG;
    if (layout == BL_PACK_1BIT && scheme != BL_BINARY) return BL_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f) return BL_ERR_INVALID_ARG;
    if (bl::pack_workspace_bytes(N * K) > bitlinear_pack_noalloc_max_scratch_bytes())
        return BL_ERR_INVALID_ARG;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    double *scratch = nullptr;
    size_t scratch_bytes = 0;
    if (bl::pack_scratch(&scratch, &scratch_bytes) != hipSuccess) {
        (void)hipGetLastError();
        return BL_ERR_DEVICE;
    }
    if (bl::pack_workspace_bytes(N * K) > scratch_bytes) return BL_ERR_INVALID_ARG;
    return launched(bl::launch_pack(W, w_dtype, N, K, scheme, layout, eps, packed, gamma,
                                    scratch, static_cast<hipStream_t>(stream)));
}

size_t bitlinear_pack_noalloc_max_scratch_bytes(void) { return bl::pack_scratch_capacity(); }

bl_status bitlinear_quant_acts(const void *x, int x_dtype, int64_t M, int64_t K, int8_t *xq,
                               float *scale, void *stream) {
    if (!x || !xq || !scale) return BL_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(scale)) return BL_ERR_INVALID_ARG;
    if (M < 0 || K < 1 || K > kMaxK || M > 2147483647LL) return BL_ERR_INVALID_ARG;
    if (!valid_dtype(x_dtype)) return BL_ERR_INVALID_ARG;
    if (M == 0) return BL_OK;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    return launched(bl::launch_quant_acts(x, x_dtype, M, K, xq, scale,
                                          static_cast<hipStream_t>(stream)));
}

bl_status bitlinear_forward(const int8_t *xq, const float *scale, const uint8_t *packed,
                            int layout, const float *gamma, int64_t M, int64_t N, int64_t K,
                            void *y, int y_dtype, int32_t *acc, void *stream) {
    return forward_impl(xq, scale, packed, layout, gamma, bl::GammaMap::single(gamma), M, N, K, y,
                        y_dtype, acc, stream);
}

bl_status bitlinear_linear(const void *x, int x_dtype, const uint8_t *packed, int layout,
                           const float *gamma, int64_t M, int64_t N, int64_t K, void *y,
                           int y_dtype, int32_t *acc, void *stream) {
    return linear_impl(x, x_dtype, packed, layout, gamma, bl::GammaMap::single(gamma), M, N, K, y,
                       y_dtype, acc, stream);
}

bl_status bitlinear_forward_segmented(const int8_t *xq, const float *scale, const uint8_t *packed,
                                      int layout, const float *gammas, const int64_t *seg_rows,
                                      int nseg, int64_t M, int64_t K, void *y, int y_dtype,
                                      int32_t *acc, void *stream) {
    bl::GammaMap gm;
    int64_t N = 0;
    if (!make_segments(gammas, seg_rows, nseg, gm, N)) return BL_ERR_INVALID_ARG;
    return forward_impl(xq, scale, packed, layout, gammas, gm, M, N, K, y, y_dtype, acc, stream);
}

bl_status bitlinear_linear_segmented(const void *x, int x_dtype, const uint8_t *packed, int layout,
                                     const float *gammas, const int64_t *seg_rows, int nseg,
                                     int64_t M, int64_t K, void *y, int y_dtype, int32_t *acc,
                                     void *stream) {
    bl::GammaMap gm;
    int64_t N = 0;
    if (!make_segments(gammas, seg_rows, nseg, gm, N)) return BL_ERR_INVALID_ARG;
    return linear_impl(x, x_dtype, packed, layout, gammas, gm, M, N, K, y, y_dtype, acc, stream);
}

bl_status bitlinear_forward_lut(const int8_t *xq, const float *scale, const uint8_t *packed,
                                int layout, const float *gamma, int64_t M, int64_t N, int64_t K,
                                void *y, int y_dtype, int32_t *acc, void *stream) {
    if (!xq || !scale || !packed || !gamma || !y) return BL_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(scale) || !aligned16(packed) || !aligned4(gamma) ||
        !aligned16(y) || (acc && !aligned16(acc)))
        return BL_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 1 || K > kMaxK || N > 2147483647LL) return BL_ERR_INVALID_ARG;
    if (!valid_layout(layout) || !valid_dtype(y_dtype)) return BL_ERR_INVALID_ARG;
    if (layout != BL_PACK_BASE3 || M > 1) return BL_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return BL_OK;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    return launched(bl::launch_forward_lut(xq, scale, packed, bl::GammaMap::single(gamma), N, K, y,
                                           y_dtype, acc, static_cast<hipStream_t>(stream)));
}

bl_status bitlinear_backward_input(const void *grad_y, int gy_dtype, const uint8_t *packed,
                                   int layout, const float *gamma, int64_t M, int64_t N,
                                   int64_t K, float *grad_x, void *stream) {
    if (!grad_y || !packed || !gamma || !grad_x) return BL_ERR_INVALID_ARG;
    if (!aligned16(grad_y) || !aligned16(packed) || !aligned4(gamma) || !aligned16(grad_x))
        return BL_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 1 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return BL_ERR_INVALID_ARG;
    if (!valid_dtype(gy_dtype) || !valid_layout(layout)) return BL_ERR_INVALID_ARG;
    if (N % 8 != 0) return BL_ERR_UNSUPPORTED;
    if (M == 0) return BL_OK;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (N == 0) return launched(bl::launch_zero_f32(grad_x, M * K, s));
    return launched(bl::launch_backward_input(grad_y, gy_dtype == BL_F32, packed, layout, gamma,
                                              M, N, K, grad_x, s));
}

bl_status bitlinear_backward_weight(const void *grad_y, const void *x, int dtype, int64_t M,
                                    int64_t N, int64_t K, float *grad_w, void *stream) {
    if (!grad_y || !x || !grad_w) return BL_ERR_INVALID_ARG;
    if (!aligned16(grad_y) || !aligned16(x) || !aligned16(grad_w)) return BL_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 1 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return BL_ERR_INVALID_ARG;
    if (!valid_dtype(dtype)) return BL_ERR_INVALID_ARG;
    if (N % 8 != 0 || K % 8 != 0) return BL_ERR_UNSUPPORTED;
    if (N == 0) return BL_OK;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (M == 0) return launched(bl::launch_zero_f32(grad_w, N * K, s));
    return launched(bl::launch_backward_weight(grad_y, x, dtype == BL_F32, M, N, K, grad_w, s));
}

bl_status bitlinear_forward_epilogue(const int8_t *xq, const float *scale, const uint8_t *packed,
                                     int layout, const float *gammas, const int64_t *seg_rows,
                                     int nseg, int64_t M, int64_t K, const void *bias,
                                     int bias_dtype, int act, const void *residual,
                                     float res_scale, void *z, void *y, int y_dtype,
                                     void *stream) {
    bl::GammaMap gm;
    int64_t N = 0;
    if (!make_segments(gammas, seg_rows, nseg, gm, N)) return BL_ERR_INVALID_ARG;
    const bl::EpilogueArgs ep{bias, bias_dtype, act, residual, res_scale, z};
    if (!valid_epilogue(ep)) return BL_ERR_INVALID_ARG;
    if (!valid_layout(layout) || !valid_dtype(y_dtype)) return BL_ERR_INVALID_ARG;
    if (M < 0 || K < 1 || K > kMaxK || M > 65535LL * 128) return BL_ERR_INVALID_ARG;
    if (M == 0) return BL_OK;
    if (!xq || !scale || !packed || !gammas || !y) return BL_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(scale) || !aligned16(packed) || !aligned4(gammas) ||
        !aligned16(y))
        return BL_ERR_INVALID_ARG;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (bl::skinny_handles(M, N, K, layout))
        return launched(bl::launch_epilogue_skinny(xq, scale, packed, layout, gm, M, N, K, y,
                                                   y_dtype, ep, s));
    const auto gemm = layout == BL_PACK_2BIT    ? bl::launch_epilogue_gemm_2bit
                      : layout == BL_PACK_BASE3 ? bl::launch_epilogue_gemm_base3
                                                : bl::launch_epilogue_gemm_1bit;
    return launched(gemm(xq, scale, packed, gm, M, N, K, y, y_dtype, ep, s));
}

bl_status bitlinear_linear_epilogue(const void *x, int x_dtype, const uint8_t *packed, int layout,
                                    const float *gammas, const int64_t *seg_rows, int nseg,
                                    int64_t M, int64_t K, const void *bias, int bias_dtype,
                                    int act, const void *residual, float res_scale, void *z,
                                    void *y, int y_dtype, void *stream) {
    bl::GammaMap gm;
    int64_t N = 0;
    if (!make_segments(gammas, seg_rows, nseg, gm, N)) return BL_ERR_INVALID_ARG;
    const bl::EpilogueArgs ep{bias, bias_dtype, act, residual, res_scale, z};
    if (!valid_epilogue(ep)) return BL_ERR_INVALID_ARG;
    if (!valid_dtype(x_dtype) || !valid_layout(layout) || !valid_dtype(y_dtype))
        return BL_ERR_INVALID_ARG;
    if (M < 0 || K < 1 || K > kMaxK) return BL_ERR_INVALID_ARG;
    if (M > bl::fused_decode_max_m()) return BL_ERR_UNSUPPORTED;
    if (M == 0) return BL_OK;
    if (!x || !packed || !gammas || !y) return BL_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(packed) || !aligned4(gammas) || !aligned16(y))
        return BL_ERR_INVALID_ARG;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    return launched(bl::launch_epilogue_linear(x, x_dtype, packed, layout, gm, M, N, K, y, y_dtype,
                                               ep, static_cast<hipStream_t>(stream)));
}

size_t bitlinear_epilogue_backward_workspace_bytes(int64_t M, int64_t N) {
    if (M < 1 || N < 1 || M > kMaxDim || N > kMaxDim) return 0;
    return (size_t)(bl::epilogue_grad_parts(M, N) * N) * sizeof(float);
}

bl_status bitlinear_epilogue_backward(const void *grad_y, int gy_dtype, const void *z, int z_dtype,
                                      int act, float res_scale, int64_t M, int64_t N, void *grad_z,
                                      int gz_dtype, float *grad_bias, void *grad_residual,
                                      void *workspace, size_t workspace_bytes, void *stream) {
    if (M < 0 || N < 0 || M > kMaxDim || N > kMaxDim) return BL_ERR_INVALID_ARG;
    if (!valid_dtype(gy_dtype) || !valid_dtype(z_dtype) || !valid_dtype(gz_dtype))
        return BL_ERR_INVALID_ARG;
    if (act < 0 || act >= bl::kActCount) return BL_ERR_INVALID_ARG;
    if (grad_residual && !std::isfinite(res_scale)) return BL_ERR_INVALID_ARG;
    if (!aligned16(grad_y) || !aligned16(z) || !aligned16(grad_z) || !aligned16(grad_bias) ||
        !aligned16(grad_residual) || !aligned16(workspace))
        return BL_ERR_INVALID_ARG;
    if (N == 0) return BL_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (M > 0) {
        if (!grad_y || (!z && act != BL_ACT_NONE)) return BL_ERR_INVALID_ARG;
        if (!grad_z && !grad_bias && !grad_residual) return BL_ERR_INVALID_ARG;
        if (grad_bias && (!workspace || workspace_bytes <
                                            bitlinear_epilogue_backward_workspace_bytes(M, N)))
            return BL_ERR_INVALID_ARG;
    } else if (!grad_bias) {
        return BL_OK;
    }
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    if (M == 0) return launched(bl::launch_zero_f32(grad_bias, N, s));
    const bl::EpilogueGradArgs a{grad_y,    z,        grad_z,  grad_residual, grad_bias,
                                 static_cast<float *>(workspace),
                                 gy_dtype,  z_dtype,  gz_dtype, act, res_scale, M, N};
    return launched(bl::launch_epilogue_backward(a, s));
}

bl_status bitlinear_forward_gated(const int8_t *xq, const float *scale, const uint8_t *packed,
                                  int layout, const float *gammas, int64_t F, int64_t M, int64_t K,
                                  const void *bias, int bias_dtype, int act, void *z,
                                  int8_t *codes, float *code_scale, void *y, int y_dtype,
                                  void *stream) {
    bl::GammaMap gm;
    const bl::GatedArgs ga{bias, bias_dtype, act, z, codes, code_scale, F};
    if (!make_pair(gammas, F, gm) || !valid_gated(ga)) return BL_ERR_INVALID_ARG;
    if (!valid_layout(layout) || !valid_dtype(y_dtype)) return BL_ERR_INVALID_ARG;
    if (M < 0 || K < 1 || K > kMaxK || M > 65535LL * 128) return BL_ERR_INVALID_ARG;
    if (M == 0) return BL_OK;
    if (!xq || !scale || !packed || !gammas || !y) return BL_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(scale) || !aligned16(packed) || !aligned4(gammas) ||
        !aligned16(y))
        return BL_ERR_INVALID_ARG;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!codes && bl::skinny_handles(M, 2 * F, K, layout))
        return launched(
            bl::launch_gated_skinny(xq, scale, packed, layout, gm, M, K, y, y_dtype, ga, s));
    const auto gemm = layout == BL_PACK_2BIT    ? bl::launch_gated_gemm_2bit
                      : layout == BL_PACK_BASE3 ? bl::launch_gated_gemm_base3
                                                : bl::launch_gated_gemm_1bit;
    return launched(gemm(xq, scale, packed, gm, M, K, y, y_dtype, ga, s));
}

bl_status bitlinear_linear_gated(const void *x, int x_dtype, const uint8_t *packed, int layout,
                                 const float *gammas, int64_t F, int64_t M, int64_t K,
                                 const void *bias, int bias_dtype, int act, void *z, void *y,
                                 int y_dtype, void *stream) {
    bl::GammaMap gm;
    const bl::GatedArgs ga{bias, bias_dtype, act, z, nullptr, nullptr, F};
    if (!make_pair(gammas, F, gm) || !valid_gated(ga)) return BL_ERR_INVALID_ARG;
    if (!valid_dtype(x_dtype) || !valid_layout(layout) || !valid_dtype(y_dtype))
        return BL_ERR_INVALID_ARG;
    if (M < 0 || K < 1 || K > kMaxK) return BL_ERR_INVALID_ARG;
    if (M > bl::fused_decode_max_m()) return BL_ERR_UNSUPPORTED;
    if (M == 0) return BL_OK;
    if (!x || !packed || !gammas || !y) return BL_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(packed) || !aligned4(gammas) || !aligned16(y))
        return BL_ERR_INVALID_ARG;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    return launched(bl::launch_gated_linear(x, x_dtype, packed, layout, gm, M, K, y, y_dtype, ga,
                                            static_cast<hipStream_t>(stream)));
}

size_t bitlinear_gated_backward_workspace_bytes(int64_t M, int64_t F) {
    if (M < 1 || F < 1 || M > kMaxDim / 2 || F > kMaxDim / 2) return 0;
    const int64_t parts = bl::gated_grad_parts(M, F);
    return parts > 1 ? (size_t)(parts * 2 * F) * sizeof(float) : 0;
}

bl_status bitlinear_gated_backward(const void *grad_y, int gy_dtype, const void *z, int z_dtype,
                                   const int8_t *codes, const float *code_scale, int act,
                                   int64_t M, int64_t F, void *grad_z, int gz_dtype,
                                   float *grad_bias, void *workspace, size_t workspace_bytes,
                                   void *stream) {
    if (M < 0 || F < 0 || M > kMaxDim / 2 || F > kMaxDim / 2) return BL_ERR_INVALID_ARG;
    if (!valid_dtype(gy_dtype) || !valid_dtype(z_dtype) || !valid_dtype(gz_dtype))
        return BL_ERR_INVALID_ARG;
    if (act < 0 || act >= bl::kActCount) return BL_ERR_INVALID_ARG;
    if (!aligned16(grad_y) || !aligned16(z) || !aligned16(codes) || !aligned16(code_scale) ||
        !aligned16(grad_z) || !aligned16(grad_bias) || !aligned16(workspace))
        return BL_ERR_INVALID_ARG;
    if (F == 0) return BL_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (M > 0) {
        if (!grad_y || (codes != nullptr) != (code_scale != nullptr) ||
            (z != nullptr) == (codes != nullptr))
            return BL_ERR_INVALID_ARG;
        if (!grad_z && !grad_bias) return BL_ERR_INVALID_ARG;
        const size_t need = grad_bias ? bitlinear_gated_backward_workspace_bytes(M, F) : 0;
        if (need > 0 && (!workspace || workspace_bytes < need)) return BL_ERR_INVALID_ARG;
    } else if (!grad_bias) {
        return BL_OK;
    }
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    if (M == 0) return launched(bl::launch_zero_f32(grad_bias, 2 * F, s));
    const bl::GatedGradArgs a{grad_y,    z,        codes,    code_scale, grad_z,
                              grad_bias, static_cast<float *>(workspace),
                              gy_dtype,  z_dtype,  gz_dtype, act,        M, F};
    return launched(bl::launch_gated_backward(a, s));
}

int64_t bitlinear_checkpoint_groups(int64_t K) { return K < 1 ? 0 : (K - 1) / bl::kCheckpointGroup + 1; }

bl_status bitlinear_checkpoint(const void *x, int x_dtype, int64_t M, int64_t K, int8_t *codes,
                               float *scale, void *stream) {
    if (M < 0 || K < 1 || M > kMaxDim || K > kMaxDim || !valid_dtype(x_dtype))
        return BL_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scale)) return BL_ERR_INVALID_ARG;
    if (M == 0) return BL_OK;
    if (!x || !codes || !scale) return BL_ERR_INVALID_ARG;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    return launched(bl::launch_checkpoint(x, x_dtype, M, K, codes, scale,
                                          static_cast<hipStream_t>(stream)));
}

bl_status bitlinear_checkpoint_restore(const int8_t *codes, const float *scale, int64_t M, int64_t K,
                                       void *y, int y_dtype, void *stream) {
    if (M < 0 || K < 1 || M > kMaxDim || K > kMaxDim || !valid_dtype(y_dtype))
        return BL_ERR_INVALID_ARG;
    if (!aligned16(codes) || !aligned16(scale) || !aligned16(y)) return BL_ERR_INVALID_ARG;
    if (M == 0) return BL_OK;
    if (!codes || !scale || !y) return BL_ERR_INVALID_ARG;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    return launched(bl::launch_checkpoint_restore(codes, scale, M, K, y, y_dtype,
                                                  static_cast<hipStream_t>(stream)));
}

size_t bitlinear_backward_weight_codes_workspace_bytes(int64_t M, int64_t N, int64_t K, int gw_dtype) {
    if (M < 1 || N < 1 || K < 1 || M > kMaxDim || N > kMaxDim || K > kMaxDim || !valid_dtype(gw_dtype))
        return 0;
    return bl::backward_weight_codes_workspace(M, N, K, gw_dtype);
}

bl_status bitlinear_backward_weight_codes(const void *grad_y, int gy_dtype, const int8_t *xq,
                                          const float *scale, int64_t M, int64_t N, int64_t K,
                                          void *grad_w, int gw_dtype, void *workspace,
                                          size_t workspace_bytes, void *stream) {
    if (M < 0 || N < 0 || K < 1 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return BL_ERR_INVALID_ARG;
    if (!valid_dtype(gy_dtype) || !valid_dtype(gw_dtype)) return BL_ERR_INVALID_ARG;
    if (!aligned16(grad_y) || !aligned16(xq) || !aligned16(scale) || !aligned16(grad_w) ||
        !aligned16(workspace))
        return BL_ERR_INVALID_ARG;
    if (N == 0) return BL_OK;
    if (!grad_w || (M > 0 && (!grad_y || !xq || !scale))) return BL_ERR_INVALID_ARG;
    const size_t need = bitlinear_backward_weight_codes_workspace_bytes(M, N, K, gw_dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return BL_ERR_INVALID_ARG;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (M == 0) return launched(bl::launch_zero(grad_w, gw_dtype, N * K, s));
    return launched(bl::launch_backward_weight_codes(grad_y, gy_dtype, xq, scale, M, N, K, grad_w,
                                                     gw_dtype, static_cast<float *>(workspace), s));
}

size_t bitlinear_backward_input_segmented_workspace_bytes(int64_t M, int64_t N, int64_t K,
                                                          int gy_dtype) {
    if (M < 1 || N < 1 || K < 1 || M > kMaxDim || N > kMaxDim / 2 || K > kMaxDim ||
        !valid_dtype(gy_dtype))
        return 0;
    return bl::backward_input_segmented_workspace(M, N, K, gy_dtype);
}

bl_status bitlinear_backward_input_segmented(const void *grad_y, int gy_dtype,
                                             const uint8_t *packed, int layout,
                                             const float *gammas, const int64_t *seg_rows, int nseg,
                                             int64_t M, int64_t K, void *grad_x, int gx_dtype,
                                             void *workspace, size_t workspace_bytes, void *stream) {
    bl::GammaMap gm;
    int64_t N = 0;
    if (!make_segments(gammas, seg_rows, nseg, gm, N)) return BL_ERR_INVALID_ARG;
    if (M < 0 || K < 1 || M > kMaxDim || N > kMaxDim / 2 || K > kMaxDim) return BL_ERR_INVALID_ARG;
    if (!valid_dtype(gy_dtype) || !valid_dtype(gx_dtype) || !valid_layout(layout))
        return BL_ERR_INVALID_ARG;
    if (M == 0) return BL_OK;
    if (!grad_y || !packed || !gammas || !grad_x) return BL_ERR_INVALID_ARG;
    if (!aligned16(grad_y) || !aligned16(packed) || !aligned4(gammas) || !aligned16(grad_x) ||
        !aligned16(workspace))
        return BL_ERR_INVALID_ARG;
    const size_t need = bitlinear_backward_input_segmented_workspace_bytes(M, N, K, gy_dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return BL_ERR_INVALID_ARG;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    return launched(bl::launch_backward_input_segmented(grad_y, gy_dtype, packed, layout, gm, M, N,
                                                        K, grad_x, gx_dtype,
                                                        static_cast<float *>(workspace),
                                                        static_cast<hipStream_t>(stream)));
}

bl_status bitlinear_block_norm(const void *h, int h_dtype, const void *block, int x_dtype,
                               float res_scale, const void *gate, int gate_kind, int post_kind,
                               const void *post_weight, const void *post_bias, float post_eps,
                               int pre_kind, const void *pre_weight, const void *pre_bias,
                               float pre_eps, int p_dtype, int64_t M, int64_t K, void *h_out,
                               void *n, int8_t *xq, float *scale, float *stats, void *stream) {
    const bl::NormSide post{post_weight, post_bias, post_kind, post_eps};
    const bl::NormSide pre{pre_weight, pre_bias, pre_kind, pre_eps};
    if (M < 0 || K < 1 || K > kMaxK || M > 2147483647LL) return BL_ERR_INVALID_ARG;
    if (!valid_dtype(h_dtype) || !valid_dtype(x_dtype) || !valid_dtype(p_dtype))
        return BL_ERR_INVALID_ARG;
    if (!valid_norm(post) || !valid_norm(pre)) return BL_ERR_INVALID_ARG;
    if (gate_kind < BL_GATE_NONE || gate_kind > BL_GATE_TOKEN || !std::isfinite(res_scale))
        return BL_ERR_INVALID_ARG;
    if (!aligned16(h) || !aligned16(block) || !aligned16(gate) || !aligned16(h_out) ||
        !aligned16(n) || !aligned16(xq) || !aligned16(scale) || !aligned16(stats))
        return BL_ERR_INVALID_ARG;
    if (M == 0) return BL_OK;
    if (!h || (gate != nullptr) != (gate_kind != BL_GATE_NONE)) return BL_ERR_INVALID_ARG;
    if (block ? !h_out : (h_out || gate || post_kind != BL_NORM_NONE)) return BL_ERR_INVALID_ARG;
    if ((xq != nullptr) != (scale != nullptr)) return BL_ERR_INVALID_ARG;
    if (pre_kind == BL_NORM_NONE ? (n || xq || !block) : (!n && !xq)) return BL_ERR_INVALID_ARG;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    const bl::BlockNormArgs a{h,       block, gate, post,  pre, h_dtype, x_dtype, p_dtype,
                              gate_kind, res_scale, M, K, h_out, n, xq, scale, stats};
    return launched(bl::launch_block_norm(a, static_cast<hipStream_t>(stream)));
}

size_t bitlinear_block_norm_backward_workspace_bytes(int64_t M, int64_t K) {
    if (M < 1 || K < 1 || M > kMaxDim || K > kMaxDim) return 0;
    return (size_t)bl::block_norm_grad_workspace(M, K) * sizeof(float);
}

bl_status bitlinear_block_norm_backward(
    const void *grad_h_out, const void *grad_n, int gn_dtype, const void *h_out, int h_dtype,
    const void *block, int x_dtype, const float *stats, float res_scale, const void *gate,
    int gate_kind, int post_kind, const void *post_weight, const void *post_bias, int pre_kind,
    const void *pre_weight, int p_dtype, int64_t M, int64_t K, void *grad_h, void *grad_block,
    void *grad_gate, float *grad_post_weight, float *grad_post_bias, float *grad_pre_weight,
    float *grad_pre_bias, void *workspace, size_t workspace_bytes, void *stream) {
    // (eps is inside the saved statistics)
    const bl::NormSide post{post_weight, post_bias, post_kind, 1.f};
    const bl::NormSide pre{pre_weight, nullptr, pre_kind, 1.f};
    if (M < 0 || K < 1 || M > kMaxDim || K > kMaxDim) return BL_ERR_INVALID_ARG;
    if (!valid_dtype(h_dtype) || !valid_dtype(x_dtype) || !valid_dtype(gn_dtype) ||
        !valid_dtype(p_dtype))
        return BL_ERR_INVALID_ARG;
    if (!valid_norm(post) || !valid_norm(pre)) return BL_ERR_INVALID_ARG;
    if (gate_kind < BL_GATE_NONE || gate_kind > BL_GATE_TOKEN || !std::isfinite(res_scale))
        return BL_ERR_INVALID_ARG;
    if (!aligned16(grad_h_out) || !aligned16(grad_n) || !aligned16(h_out) || !aligned16(block) ||
        !aligned16(stats) || !aligned16(gate) || !aligned16(grad_h) || !aligned16(grad_block) ||
        !aligned16(grad_gate) || !aligned16(grad_post_weight) || !aligned16(grad_post_bias) ||
        !aligned16(grad_pre_weight) || !aligned16(grad_pre_bias) || !aligned16(workspace))
        return BL_ERR_INVALID_ARG;
    if (post_kind == BL_NORM_NONE && (grad_post_weight || grad_post_bias))
        return BL_ERR_INVALID_ARG;
    if (pre_kind == BL_NORM_NONE && (grad_pre_weight || grad_pre_bias)) return BL_ERR_INVALID_ARG;
    if (gate_kind == BL_GATE_NONE && grad_gate) return BL_ERR_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (M == 0) {
        float *const sums[5] = {grad_post_weight, grad_post_bias, grad_pre_weight, grad_pre_bias,
                                gate_kind == BL_GATE_CHANNEL ? static_cast<float *>(grad_gate)
                                                             : nullptr};
        for (float *p : sums) {
            if (!p) continue;
            bl_status st = device_ok();
            if (st == BL_OK) st = launched(bl::launch_zero_f32(p, K, s));
            if (st != BL_OK) return st;
        }
        return BL_OK;
    }
    if (!h_out || !stats || !grad_h) return BL_ERR_INVALID_ARG;
    if ((grad_n != nullptr) != (pre_kind != BL_NORM_NONE)) return BL_ERR_INVALID_ARG;
    if ((gate != nullptr) != (gate_kind != BL_GATE_NONE)) return BL_ERR_INVALID_ARG;
    if (!grad_n && !block) return BL_ERR_INVALID_ARG;
    if (!block && (gate || post_kind != BL_NORM_NONE || grad_block)) return BL_ERR_INVALID_ARG;
    if (!workspace ||
        workspace_bytes < bitlinear_block_norm_backward_workspace_bytes(M, K))
        return BL_ERR_INVALID_ARG;
    bl_status st = device_ok();
    if (st != BL_OK) return st;
    const bl::BlockNormGradArgs a{grad_h_out, grad_n, h_out, block, gate, stats, post, pre,
                                  h_dtype, x_dtype, gn_dtype, p_dtype, gate_kind, res_scale, M, K,
                                  grad_h, grad_block, grad_gate, grad_post_weight, grad_post_bias,
                                  grad_pre_weight, grad_pre_bias, static_cast<float *>(workspace)};
    return launched(bl::launch_block_norm_backward(a, s));
}

int bitlinear_forward_plan(int64_t M, int64_t N, int64_t K, int layout, int y_dtype, int fused,
                           char *buf, size_t len) {
    if (M < 0 || N < 0 || K < 1 || K > kMaxK || N > 2147483647LL) return -1;
    if (!valid_layout(layout) || !valid_dtype(y_dtype)) return -1;
    if (fused ? M > bl::fused_decode_max_m() : M > 65535LL * 128) return -1;
    bl::PlanSink sink;
    if (M > 0 && N > 0) {
        // stand-in addresses: with a sink installed nothing is launched and no
        // pointer is dereferenced, only offset
        const uintptr_t fake = 4096;
        auto *xq = reinterpret_cast<const int8_t *>(fake);
        auto *sc = reinterpret_cast<const float *>(fake);
        auto *pk = reinterpret_cast<const uint8_t *>(fake);
        const bl::GammaMap gm = bl::GammaMap::single(sc);
        void *y = reinterpret_cast<void *>(fake);
        bl::t_plan = &sink;
        if (fused)
            (void)bl::launch_linear_decode(y, BL_BF16, pk, layout, gm, M, N, K, y, y_dtype,
                                           nullptr, nullptr);
        else if (bl::skinny_handles(M, N, K, layout))
            (void)bl::launch_forward_skinny(xq, sc, pk, layout, gm, M, N, K, y, y_dtype, nullptr,
                                            nullptr);
        else
            (void)bl::launch_forward_gemm(xq, sc, pk, layout, gm, M, N, K, y, y_dtype, nullptr,
                                          nullptr);
        bl::t_plan = nullptr;
    }
    if (buf && len > 0) {
        const size_t n = sink.text.size() < len - 1 ? sink.text.size() : len - 1;
        std::memcpy(buf, sink.text.data(), n);
        buf[n] = '\0';
    }
    return sink.launches;
}

const char *bitlinear_status_string(int status) {
    switch (status) {
        case BL_OK: return "ok";
        case BL_ERR_INVALID_ARG: return "invalid argument";
        case BL_ERR_UNSUPPORTED: return "unsupported";
        case BL_ERR_DEVICE: return "device error (no gfx950 GPU, or a launch failed)";
        default: return "unknown status";
    }
}

int bitlinear_version(void) { return (1 << 16) | 3; }

const char *bitlinear_source_hash(void) { return BL_SOURCE_HASH; }

}  // extern "C"
