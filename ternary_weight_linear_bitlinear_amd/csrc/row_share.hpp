// Rows of a tensor split over the threads of a workgroup, held in registers: the
// loads and stores of the norm and epilogue-gradient kernels.
#pragma once

#include <type_traits>

#include "device_util.hpp"

namespace bl {

template <typename T>
__device__ __forceinline__ void put(T *p, int64_t i, float v) {
    if constexpr (sizeof(T) == 4) p[i] = v;
    else p[i] = (T)f32_to_bf16_rne(v);
}

// One thread's share of a row: chunk j, element e is element index(j, e) of the
// row, below K where valid.
template <int J, bool VEC>
struct Share {
    int K, tid, T;
    __device__ __forceinline__ int index(int j, int e) const {
        return VEC ? (j * T + tid) * 8 + e : (j * 8 + e) * T + tid;
    }
    __device__ __forceinline__ bool valid(int j, int e) const { return index(j, e) < K; }
};
// A share of a tensor's row as loaded; elements past K read a valid address and
// are zeroed when widened.
template <typename T, int J, bool VEC> struct RowRegs;
template <typename T, int J> struct RowRegs<T, J, true> {
    Raw8<T> raw[J];
    __device__ __forceinline__ void load(const T *row, const Share<J, true> &sh) {
#pragma unroll
        for (int j = 0; j < J; ++j) raw[j].load(row + (sh.valid(j, 0) ? sh.index(j, 0) : 0));
    }
    __device__ __forceinline__ void widen(int j, const Share<J, true> &sh, float (&v)[8]) const {
        raw[j].widen(v);
        const bool ok = sh.valid(j, 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = ok ? v[e] : 0.f;
    }
};
template <typename T, int J> struct RowRegs<T, J, false> {
    T raw[J][8];
    __device__ __forceinline__ void load(const T *row, const Share<J, false> &sh) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) raw[j][e] = row[sh.valid(j, e) ? sh.index(j, e) : 0];
    }
    __device__ __forceinline__ void widen(int j, const Share<J, false> &sh, float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = sh.valid(j, e) ? Elem<T>::get(&raw[j][e], 0) : 0.f;
    }
};
template <typename T, int J, bool VEC>
__device__ __forceinline__ void store_share(T *row, int j, const Share<J, VEC> &sh, const float (&v)[8]) {
    if constexpr (VEC) {
        if (!sh.valid(j, 0)) return;
        T *p = row + sh.index(j, 0);
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bf16x2 q = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
                w[i] = __builtin_bit_cast(uint32_t, q);
            }
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (sh.valid(j, e)) put(row, sh.index(j, e), v[e]);
    }
}

// Calls go(float or uint16_t pointer) by a tensor's type.
template <typename F>
hipError_t typed(int dtype, F go) {
    return dtype == kF32 ? go(static_cast<float *>(nullptr)) : go(static_cast<uint16_t *>(nullptr));
}
template <typename T> using Pointee = std::remove_pointer_t<T>;

}  // namespace bl
