// Epilogue of the products beyond the dequant: bias, activation and residual.
//   z = gamma * scale / 127 * acc + bias
//   y = act(z) + res_scale * residual
// computed in fp32 from the exact INT32 sums and rounded once to y's type
// (and once to z's, where the pre-activation is asked for).
#pragma once

#include <stdint.h>

#include "activation.hpp"
#include "bl_internal.hpp"
#include "device_util.hpp"

namespace bl {

// The plain dequant epilogue: the products store gamma * scale / 127 * acc
// (and the sums) themselves.
struct NoEpilogue {
    static constexpr bool kActive = false;
    NoEpilogue from_col(int64_t) const { return {}; }
};

// Operands of the extended epilogue, column 0 being the launch's first output
// column. residual and z are laid out and typed as y.
template <typename YT>
struct Epilogue {
    static constexpr bool kActive = true;
    const void *bias;    // [N] fp32, or bf16 when bias_bf16; NULL = none
    const YT *residual;  // NULL = none; may be y itself
    YT *z;               // NULL = not stored
    float res_scale;
    int act;
    int bias_bf16;

    // the same operands seen from output column `off` on
    Epilogue from_col(int64_t off) const {
        Epilogue e = *this;
        if (bias)
            e.bias = bias_bf16 ? static_cast<const void *>(static_cast<const uint16_t *>(bias) + off)
                               : static_cast<const void *>(static_cast<const float *>(bias) + off);
        if (residual) e.residual = residual + off;
        if (z) e.z = z + off;
        return e;
    }

#if defined(__HIPCC__)
    __device__ __forceinline__ static float widen(float v) { return v; }
    __device__ __forceinline__ static float widen(uint16_t v) { return bf16_bits_to_f32(v); }
    __device__ __forceinline__ static YT narrow(float v) {
        if constexpr (sizeof(YT) == 4) return v;
        else return (YT)f32_to_bf16_rne(v);
    }
    __device__ __forceinline__ float bias_at(int64_t n) const {
        return bias_bf16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(bias)[n])
                         : static_cast<const float *>(bias)[n];
    }

    // Up to four consecutive outputs n .. n + 3 (those below N) of token m
    // from their dequantised products v; y, z and residual have row stride ld.
    __device__ __forceinline__ void store4(const float (&v)[4], int64_t m, int64_t n, int64_t N,
                                           int64_t ld, YT *y) const {
        const int64_t at = m * ld + n;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (n + e >= N) continue;
            const float zv = bias ? v[e] + bias_at(n + e) : v[e];
            float a = activate(zv, act);
            if (residual) a = __builtin_fmaf(res_scale, widen(residual[at + e]), a);
            if (z) z[at + e] = narrow(zv);
            y[at + e] = narrow(a);
        }
    }
#endif
};

template <typename YT>
Epilogue<YT> make_epilogue(const EpilogueArgs &a) {
    return Epilogue<YT>{a.bias, static_cast<const YT *>(a.residual), static_cast<YT *>(a.z),
                        a.res_scale, a.act, a.bias_dtype == kBF16};
}

}  // namespace bl
