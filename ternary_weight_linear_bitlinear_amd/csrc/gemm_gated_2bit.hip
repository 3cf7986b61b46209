// The tiled products of 2-bit rows with the gated epilogue (gemm_core.hpp). One file per
// layout, so that they build in parallel.
#include "gemm_core.hpp"

namespace bl {

hipError_t launch_gated_gemm_2bit(const int8_t *xq, const float *scale, const uint8_t *packed,
                                  const GammaMap &gamma, int64_t M, int64_t K, void *y, int y_dtype,
                                  const GatedArgs &ga, hipStream_t stream) {
    const int64_t N = 2 * ga.F, rb = row_bytes_of(kLayout2Bit, K);
    if (y_dtype == kF32)
        return launch_gemm_t<kLayout2Bit>(xq, scale, packed, gamma, M, N, K, static_cast<float *>(y),
                                         nullptr, stream, make_gated<float>(ga, rb));
    return launch_gemm_t<kLayout2Bit>(xq, scale, packed, gamma, M, N, K, static_cast<uint16_t *>(y),
                                     nullptr, stream, make_gated<uint16_t>(ga, rb));
}

}  // namespace bl
