// The weight-streaming decode products with the plain dequant epilogue
// (skinny_core.hpp), and the rule for which batches they take.
#include "skinny_core.hpp"

namespace bl {
namespace {

template <int LAYOUT, typename XT>
hipError_t launch_linear_x(const XT *x, const uint8_t *packed, const GammaMap &gamma, int64_t M,
                           int64_t N, int64_t K, void *y, int y_dtype, int32_t *acc,
                           hipStream_t s) {
    if (y_dtype == kF32)
        return launch_linear_t<LAYOUT>(x, packed, gamma, M, N, K, static_cast<float *>(y), acc, s,
                                       NoEpilogue{});
    return launch_linear_t<LAYOUT>(x, packed, gamma, M, N, K, static_cast<uint16_t *>(y), acc, s,
                                   NoEpilogue{});
}

template <int LAYOUT>
hipError_t skinny_y(const int8_t *xq, const float *scale, const uint8_t *packed,
                    const GammaMap &gamma, int64_t M, int64_t N, int64_t K, void *y, int y_dtype,
                    int32_t *acc, hipStream_t stream) {
    if (y_dtype == kF32)
        return launch_skinny_l<LAYOUT>(xq, scale, packed, gamma, M, N, K, static_cast<float *>(y),
                                       acc, stream, NoEpilogue{});
    return launch_skinny_l<LAYOUT>(xq, scale, packed, gamma, M, N, K, static_cast<uint16_t *>(y),
                                   acc, stream, NoEpilogue{});
}

template <int LAYOUT>
hipError_t linear_xy(const void *x, int x_dtype, const uint8_t *packed, const GammaMap &gamma,
                     int64_t M, int64_t N, int64_t K, void *y, int y_dtype, int32_t *acc,
                     hipStream_t stream) {
    if (x_dtype == kF32)
        return launch_linear_x<LAYOUT>(static_cast<const float *>(x), packed, gamma, M, N, K, y,
                                       y_dtype, acc, stream);
    return launch_linear_x<LAYOUT>(static_cast<const uint16_t *>(x), packed, gamma, M, N, K, y,
                                   y_dtype, acc, stream);
}

}  // namespace

hipError_t launch_forward_skinny(const int8_t *xq, const float *scale, const uint8_t *packed,
                                 int layout, const GammaMap &gamma, int64_t M, int64_t N, int64_t K,
                                 void *y, int y_dtype, int32_t *acc, hipStream_t stream) {
    switch (layout) {
        case kLayout2Bit:
            return skinny_y<kLayout2Bit>(xq, scale, packed, gamma, M, N, K, y, y_dtype, acc, stream);
        case kLayoutBase3:
            return skinny_y<kLayoutBase3>(xq, scale, packed, gamma, M, N, K, y, y_dtype, acc, stream);
        default:
            return skinny_y<kLayout1Bit>(xq, scale, packed, gamma, M, N, K, y, y_dtype, acc, stream);
    }
}

int64_t fused_decode_max_m() { return kFusedMaxM; }

// Batches above 16 tokens stream the weights once per 16-token chunk (all
// chunks in one launch). That beats the tiled GEMM for a few chunks: with few
// token tiles the GEMM keeps few blocks busy, each walking all of K, and long
// rows (K >= 8192) favour the chunks further. Crossovers measured on MI355X
// with the weights streamed from HBM (K = 4096 and 11008, N = 4096 to 32768):
// 2-bit and 1-bit up to 3 chunks at any N, 6 at N <= 8192, 8 for long rows at
// N <= 16384; base-3, whose decode costs more per byte, up to 3 chunks at
// N <= 16384 and 5 at N <= 4096.
bool skinny_handles(int64_t M, int64_t N, int64_t K, int layout) {
    if (M <= kSkinnyMaxM) return true;
    const int64_t chunks = (M + kSkinnyMaxM - 1) / kSkinnyMaxM;
    if (layout == kLayoutBase3) return (N <= 4096 && chunks <= 5) || (N <= 16384 && chunks <= 3);
    return chunks <= 3 || (N <= 8192 && chunks <= 6) || (K >= 8192 && N <= 16384 && chunks <= 8);
}

hipError_t launch_linear_decode(const void *x, int x_dtype, const uint8_t *packed, int layout,
                                const GammaMap &gamma, int64_t M, int64_t N, int64_t K, void *y,
                                int y_dtype, int32_t *acc, hipStream_t stream) {
    switch (layout) {
        case kLayout2Bit:
            return linear_xy<kLayout2Bit>(x, x_dtype, packed, gamma, M, N, K, y, y_dtype, acc, stream);
        case kLayoutBase3:
            return linear_xy<kLayoutBase3>(x, x_dtype, packed, gamma, M, N, K, y, y_dtype, acc, stream);
        default:
            return linear_xy<kLayout1Bit>(x, x_dtype, packed, gamma, M, N, K, y, y_dtype, acc, stream);
    }
}

}  // namespace bl
