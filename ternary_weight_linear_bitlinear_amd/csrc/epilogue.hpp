// Epilogue of the products beyond the dequant: bias, activation and residual.
//   z = gamma * scale / 127 * acc + bias
//   y = act(z) + res_scale * residual
// computed in fp32 from the exact INT32 sums and rounded once to y's type
// (and once to z's, where the pre-activation is asked for).
#pragma once

#include <stdint.h>

#include <type_traits>

#include "activation.hpp"
#include "bl_internal.hpp"
#include "device_util.hpp"

namespace bl {

// The plain dequant epilogue: the products store gamma * scale / 127 * acc
// (and the sums) themselves.
struct NoEpilogue {
    static constexpr bool kActive = false, kGated = false;
    static constexpr int kPair = 1;  // weight rows behind an output column
    NoEpilogue from_col(int64_t) const { return {}; }
};

// Operands of the extended epilogue, column 0 being the launch's first output
// column. residual and z are laid out and typed as y.
template <typename YT>
struct Epilogue {
    static constexpr bool kActive = true, kGated = false;
    static constexpr int kPair = 1;
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

    // bias of columns n .. n + C - 1 (0 past N, and without a bias); n is a
    // multiple of 4, the vector 16-byte aligned
    template <int C>
    __device__ __forceinline__ void load_bias(int64_t n, int64_t N, float (&b)[C]) const {
        if (bias && n + C <= N) {
            if (bias_bf16) Epilogue<uint16_t>::load(static_cast<const uint16_t *>(bias) + n, b);
            else Epilogue<float>::load(static_cast<const float *>(bias) + n, b);
            return;
        }
#pragma unroll
        for (int e = 0; e < C; ++e) b[e] = bias && n + e < N ? bias_at(n + e) : 0.f;
    }
    // pieces of four bf16 or fp32 values, and of eight bf16, as loaded and as stored
    __device__ __forceinline__ static void unpack(const uint2 &q, float (&v)[4]) {
        const uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            v[e] = __uint_as_float(w[e / 2] << 16);
            v[e + 1] = __uint_as_float(w[e / 2] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ static void unpack(const uint4 &q, float (&v)[8]) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            v[e] = __uint_as_float(w[e / 2] << 16);
            v[e + 1] = __uint_as_float(w[e / 2] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ static void unpack(const uint4 &q, float (&v)[4]) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(w[e]);
    }
    template <int C>
    __device__ __forceinline__ static void load(const YT *p, float (&v)[C]) {  // C * sizeof(YT) aligned
        if constexpr (sizeof(YT) == 4) {
#pragma unroll
            for (int e = 0; e < C; e += 4) {
                const float4 q = *reinterpret_cast<const float4 *>(p + e);
                v[e] = q.x; v[e + 1] = q.y; v[e + 2] = q.z; v[e + 3] = q.w;
            }
        } else if constexpr (C == 8) {
            unpack(*reinterpret_cast<const uint4 *>(p), v);
        } else {
            unpack(*reinterpret_cast<const uint2 *>(p), v);
        }
    }
    template <int C>
    __device__ __forceinline__ static void store(YT *p, const float (&v)[C]) {
        if constexpr (sizeof(YT) == 4) {
#pragma unroll
            for (int e = 0; e < C; e += 4)
                *reinterpret_cast<float4 *>(p + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        } else {
            uint32_t w[C / 2];
#pragma unroll
            for (int e = 0; e < C; e += 2) {
                const bf16x2 q = {(__bf16)v[e], (__bf16)v[e + 1]};
                w[e / 2] = __builtin_bit_cast(uint32_t, q);
            }
            if constexpr (C == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
            else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        }
    }

    // residual of C consecutive outputs (0 past N, and without one); `at` = the
    // token's row offset + n in y, z and residual. vec: all C are below N and
    // at * sizeof(YT) is aligned to C outputs.
    template <int C>
    __device__ __forceinline__ void load_residual(int64_t at, int64_t n, int64_t N, bool vec,
                                                  float (&r)[C]) const {
        if (!residual) {
#pragma unroll
            for (int e = 0; e < C; ++e) r[e] = 0.f;
        } else if (vec) {
            load(residual + at, r);
        } else {
#pragma unroll
            for (int e = 0; e < C; ++e) r[e] = n + e < N ? widen(residual[at + e]) : 0.f;
        }
    }

    // C consecutive outputs n .. n + C - 1 (those below N) of one token from
    // their dequantised products v, bias b and residual r.
    template <int C>
    __device__ __forceinline__ void finish(float (&v)[C], const float (&b)[C], const float (&r)[C],
                                           int64_t at, int64_t n, int64_t N, bool vec, YT *y) const {
        if (bias) {
#pragma unroll
            for (int e = 0; e < C; ++e) v[e] += b[e];
        }
        if (z) put(z, v, at, n, N, vec);
        activate_all(v, act);
        if (residual) {
#pragma unroll
            for (int e = 0; e < C; ++e) v[e] = __builtin_fmaf(res_scale, r[e], v[e]);
        }
        put(y, v, at, n, N, vec);
    }
    template <int C>
    __device__ __forceinline__ static void put(YT *p, const float (&v)[C], int64_t at, int64_t n,
                                               int64_t N, bool vec) {
        if (vec) {
            store(p + at, v);
            return;
        }
#pragma unroll
        for (int e = 0; e < C; ++e)
            if (n + e < N) p[at + e] = narrow(v[e]);
    }
#endif
};

// Operands of the gated epilogue. The packed matrix is a stack of two, gate rows
// 0 .. F - 1 and up rows F .. 2F - 1, and output column f is
//   z_h = gamma_h * scale / 127 * acc[h F + f] + bias[h F + f],  h = 0 (gate), 1 (up)
//   y[f] = act(z_0) * z_1
// in fp32, rounded once to y's type; z [M, 2F] is laid out as the stack's output.
// A launch's N counts weight rows, two for each output column; how a tile of them
// is dealt to the halves is up to the kernel (both halves of a column in one tile).
template <typename YT>
struct GatedEpilogue {
    static constexpr bool kActive = true, kGated = true;
    static constexpr int kPair = 2;
    const void *bias;   // [2F] fp32, or bf16 when bias_bf16; NULL = none
    YT *z;              // NULL = not stored
    int8_t *codes;      // [2M, F]: z in 8 bits, rows 2m (gate) and 2m + 1 (up); NULL = not kept
    float *code_scale;  // [2M, groups]
    int64_t F, groups;  // columns in all; checkpoint groups of a row
    int64_t up;         // bytes from a gate row to its up row
    int64_t col0;       // the launch's first output column
    int act;
    int bias_bf16;

    // the same operands seen from weight row `off` of the launch on
    GatedEpilogue from_col(int64_t off) const {
        GatedEpilogue e = *this;
        e.col0 += off / 2;
        return e;
    }

#if defined(__HIPCC__)
    using Ep = Epilogue<YT>;
    __device__ __forceinline__ float bias_at(int64_t n) const {
        return bias_bf16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(bias)[n])
                         : static_cast<const float *>(bias)[n];
    }
    // Bias of columns n .. n + C - 1 of half h (0 past F, and without a bias); n is a
    // multiple of C, counted over all columns.
    template <int C>
    __device__ __forceinline__ void load_bias(int h, int64_t n, float (&b)[C]) const {
        if (bias && n + C <= F && F % C == 0) {
            if (bias_bf16) Epilogue<uint16_t>::load(static_cast<const uint16_t *>(bias) + h * F + n, b);
            else Epilogue<float>::load(static_cast<const float *>(bias) + h * F + n, b);
            return;
        }
#pragma unroll
        for (int e = 0; e < C; ++e) b[e] = bias && n + e < F ? bias_at(h * F + n + e) : 0.f;
    }
    // C consecutive outputs of token m from both halves' dequantised products g and u,
    // which leave as the pre-activations: columns n .. n + C - 1 of all (those below F);
    // yt[e] is column n + e of y. vec: all C are below F, and F and yt are aligned to C
    // outputs.
    template <int C>
    __device__ __forceinline__ void finish(float (&g)[C], float (&u)[C], const float (&bg)[C],
                                           const float (&bu)[C], int64_t m, int64_t n, bool vec,
                                           YT *yt) const {
        if (bias) {
#pragma unroll
            for (int e = 0; e < C; ++e) {
                g[e] += bg[e];
                u[e] += bu[e];
            }
        }
        if (z) {
            Ep::put(z + m * 2 * F + n, g, 0, n, F, vec);
            Ep::put(z + m * 2 * F + F + n, u, 0, n, F, vec);
        }
        float v[C];
#pragma unroll
        for (int e = 0; e < C; ++e) v[e] = g[e];
        activate_all(v, act);
#pragma unroll
        for (int e = 0; e < C; ++e) v[e] *= u[e];
        Ep::put(yt, v, 0, n, F, vec);
    }
#endif
};

// How a product's kernel takes y: the plain epilogue never reads what it writes,
// the extended one may be given y as its residual.
template <typename YT, typename E>
using OutPtr = std::conditional_t<E::kActive, YT *, YT *__restrict__>;

template <typename YT>
Epilogue<YT> make_epilogue(const EpilogueArgs &a) {
    return Epilogue<YT>{a.bias, static_cast<const YT *>(a.residual), static_cast<YT *>(a.z),
                        a.res_scale, a.act, a.bias_dtype == kBF16};
}
template <typename YT>
GatedEpilogue<YT> make_gated(const GatedArgs &a, int64_t row_bytes) {
    return GatedEpilogue<YT>{a.bias, static_cast<YT *>(a.z), a.codes, a.code_scale, a.F,
                             checkpoint_groups(a.F), a.F * row_bytes, 0, a.act,
                             a.bias_dtype == kBF16};
}

}  // namespace bl
