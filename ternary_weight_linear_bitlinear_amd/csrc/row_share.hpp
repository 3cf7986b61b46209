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

// One thread's share of a row of K elements: J chunks of eight consecutive ones,
// T chunks apart. VEC: K % 8 == 0, every row and chunk 16-byte aligned. Otherwise
// (K >= 8) rows begin at any element: chunks move as unaligned 16-byte accesses,
// which the hardware splits where they cross a cache line, and the chunk that would
// run past the row's end begins eight elements before it instead, overlapping its
// neighbour; it owns only what is past the neighbour's share (element skip(j) on).
// No load has a branch or a select behind it, so the loads of several tensors
// stay in flight together. (333 x 5001 LayerNorm: 12.5 us with single elements
// throughout, 10.8 us with the end's elements one by one,
// 9.3 us this way.)
template <int J, bool VEC>
struct Share {
    int K, tid, T;
    __device__ __forceinline__ int chunk(int j) const { return (j * T + tid) * 8; }
    __device__ __forceinline__ int start(int j) const {  // the element that chunk j is loaded from
        const int k = chunk(j);
        return VEC ? (k < K ? k : 0) : (k < K - 8 ? k : K - 8);
    }
    __device__ __forceinline__ int skip(int j) const {  // 8 or more: the chunk owns nothing
        return VEC ? (chunk(j) < K ? 0 : 8) : chunk(j) - start(j);
    }
};
struct __attribute__((packed, aligned(1))) Bytes8 { uint32_t w[2]; };
struct __attribute__((packed, aligned(2))) Halves8 { uint32_t w[4]; };
struct __attribute__((packed, aligned(4))) Floats8 { float v[8]; };
__device__ __forceinline__ void load_any(const uint16_t *p, Raw8<uint16_t> &r) {
    const Halves8 h = *reinterpret_cast<const Halves8 *>(p);
    r.a = make_uint4(h.w[0], h.w[1], h.w[2], h.w[3]);
}
__device__ __forceinline__ void load_any(const float *p, Raw8<float> &r) {
    const Floats8 f = *reinterpret_cast<const Floats8 *>(p);
    r.a = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
    r.b = make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
}
template <typename T, int J, bool VEC>
__device__ __forceinline__ void load_chunk(const T *row, int j, const Share<J, VEC> &sh, Raw8<T> &r) {
    if constexpr (VEC) r.load(row + sh.start(j));
    else load_any(row + sh.start(j), r);
}
// Zeroes what the chunk does not own. Only waves that hold a row's end, or nothing of
// it, spend instructions on it: on short rows these kernels are bound by the vector
// unit.
template <int J, bool VEC>
__device__ __forceinline__ void clear_past(int j, const Share<J, VEC> &sh, float (&v)[8]) {
    const int skip = sh.skip(j);
    if (skip == 0) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = !VEC && e >= skip ? v[e] : 0.f;
}
// A share of a tensor's row.
template <typename T, int J, bool VEC>
struct RowRegs {
    Raw8<T> raw[J];
    __device__ __forceinline__ void load(const T *row, const Share<J, VEC> &sh) {
#pragma unroll
        for (int j = 0; j < J; ++j) load_chunk(row, j, sh, raw[j]);
    }
    // Chunk j in fp32, zero where it owns nothing.
    __device__ __forceinline__ void widen(int j, const Share<J, VEC> &sh, float (&v)[8]) const {
        raw[j].widen(v);
        clear_past(j, sh, v);
    }
};
template <typename T, int J, bool VEC>
__device__ __forceinline__ void store_share(T *row, int j, const Share<J, VEC> &sh, const float (&v)[8]) {
    T *p = row + sh.start(j);
    const int skip = sh.skip(j);
    if (skip == 0) {
        uint32_t w[4];
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bf16x2 q = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
                w[i] = __builtin_bit_cast(uint32_t, q);
            }
            if constexpr (VEC) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
            else *reinterpret_cast<Halves8 *>(p) = Halves8{{w[0], w[1], w[2], w[3]}};
        } else if constexpr (VEC) {
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<Floats8 *>(p) = Floats8{{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]}};
        }
    } else if constexpr (!VEC) {
#pragma unroll
        for (int e = 1; e < 8; ++e)
            if (e >= skip) put(p, e, v[e]);
    }
}

// Calls go(float or uint16_t pointer) by a tensor's type.
template <typename F>
hipError_t typed(int dtype, F go) {
    return dtype == kF32 ? go(static_cast<float *>(nullptr)) : go(static_cast<uint16_t *>(nullptr));
}
template <typename T> using Pointee = std::remove_pointer_t<T>;

}  // namespace bl
