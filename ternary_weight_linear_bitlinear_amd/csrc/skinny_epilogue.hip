// The weight-streaming decode products with bias, activation and residual in
// the epilogue (skinny_core.hpp).
#include "skinny_core.hpp"

#include <type_traits>

namespace bl {
namespace {

template <typename F>
hipError_t with_layout(int layout, F go) {
    switch (layout) {
        case kLayout2Bit: return go(std::integral_constant<int, kLayout2Bit>{});
        case kLayoutBase3: return go(std::integral_constant<int, kLayoutBase3>{});
        default: return go(std::integral_constant<int, kLayout1Bit>{});
    }
}

}  // namespace

hipError_t launch_epilogue_skinny(const int8_t *xq, const float *scale, const uint8_t *packed,
                                  int layout, const GammaMap &gamma, int64_t M, int64_t N,
                                  int64_t K, void *y, int y_dtype, const EpilogueArgs &ep,
                                  hipStream_t stream) {
    return with_layout(layout, [&](auto layout_c) {
        constexpr int L = decltype(layout_c)::value;
        if (y_dtype == kF32)
            return launch_skinny_l<L>(xq, scale, packed, gamma, M, N, K, static_cast<float *>(y),
                                      nullptr, stream, make_epilogue<float>(ep));
        return launch_skinny_l<L>(xq, scale, packed, gamma, M, N, K, static_cast<uint16_t *>(y),
                                  nullptr, stream, make_epilogue<uint16_t>(ep));
    });
}

hipError_t launch_epilogue_linear(const void *x, int x_dtype, const uint8_t *packed, int layout,
                                  const GammaMap &gamma, int64_t M, int64_t N, int64_t K, void *y,
                                  int y_dtype, const EpilogueArgs &ep, hipStream_t stream) {
    return with_layout(layout, [&](auto layout_c) {
        constexpr int L = decltype(layout_c)::value;
        auto typed = [&](auto *xt) {
            if (y_dtype == kF32)
                return launch_linear_t<L>(xt, packed, gamma, M, N, K, static_cast<float *>(y),
                                          nullptr, stream, make_epilogue<float>(ep));
            return launch_linear_t<L>(xt, packed, gamma, M, N, K, static_cast<uint16_t *>(y),
                                      nullptr, stream, make_epilogue<uint16_t>(ep));
        };
        if (x_dtype == kF32) return typed(static_cast<const float *>(x));
        return typed(static_cast<const uint16_t *>(x));
    });
}

}  // namespace bl
