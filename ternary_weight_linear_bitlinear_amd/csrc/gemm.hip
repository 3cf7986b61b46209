// The tiled INT8 matrix-core products with the plain dequant epilogue
// (gemm_core.hpp): bitlinear_forward above the decode batches.
#include "gemm_core.hpp"

namespace bl {

hipError_t launch_forward_gemm(const int8_t *xq, const float *scale, const uint8_t *packed,
                               int layout, const GammaMap &gamma, int64_t M, int64_t N, int64_t K,
                               void *y, int y_dtype, int32_t *acc, hipStream_t stream) {
    if (M > (int64_t)2147483647 || N > (int64_t)2147483647) return hipErrorInvalidValue;
    auto go = [&](auto layout_c) {
        constexpr int L = decltype(layout_c)::value;
        if (y_dtype == kF32)
            return launch_gemm_t<L>(xq, scale, packed, gamma, M, N, K, static_cast<float *>(y),
                                    acc, stream, NoEpilogue{});
        return launch_gemm_t<L>(xq, scale, packed, gamma, M, N, K, static_cast<uint16_t *>(y),
                                acc, stream, NoEpilogue{});
    };
    switch (layout) {
        case kLayout2Bit: return go(std::integral_constant<int, kLayout2Bit>{});
        case kLayoutBase3: return go(std::integral_constant<int, kLayoutBase3>{});
        default: return go(std::integral_constant<int, kLayout1Bit>{});
    }
}

}  // namespace bl
