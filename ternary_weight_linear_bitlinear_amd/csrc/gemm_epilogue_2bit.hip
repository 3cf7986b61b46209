// The tiled products of 2-bit rows with bias, activation and residual in the
// epilogue (gemm_core.hpp). One file per layout, so that they build in parallel.
#include "gemm_core.hpp"

namespace bl {

hipError_t launch_epilogue_gemm_2bit(const int8_t *xq, const float *scale, const uint8_t *packed,
                                     const GammaMap &gamma, int64_t M, int64_t N, int64_t K, void *y,
                                     int y_dtype, const EpilogueArgs &ep, hipStream_t stream) {
    if (y_dtype == kF32)
        return launch_gemm_t<kLayout2Bit>(xq, scale, packed, gamma, M, N, K, static_cast<float *>(y),
                                 nullptr, stream, make_epilogue<float>(ep));
    return launch_gemm_t<kLayout2Bit>(xq, scale, packed, gamma, M, N, K, static_cast<uint16_t *>(y),
                             nullptr, stream, make_epilogue<uint16_t>(ep));
}

}  // namespace bl
