// What the backward products share: matrix-core operand types, packed codes as bf16
// and fp32 values in bf16 pieces.
#pragma once

#include "device_util.hpp"

namespace bl {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

// Four codes of one 2-bit field (bytes u = c + 1 in 0..2) to four bf16 values
// -1 / 0 / +1 (0xBF80 / 0x0000 / 0x3F80) in two dwords. The byte permute picks
// table bytes by selector: selector (u, u + 4) yields (low byte, high byte).
template <uint32_t kLo, uint32_t kHi>
__device__ __forceinline__ void field_to_16(uint32_t f, uint32_t &d0, uint32_t &d1) {
    const uint32_t f4 = f + 0x04040404u;
    const uint32_t s0 = __builtin_amdgcn_perm(f4, f, 0x05010400u);  // u0, u0+4, u1, u1+4
    const uint32_t s1 = __builtin_amdgcn_perm(f4, f, 0x07030602u);  // u2, u2+4, u3, u3+4
    d0 = __builtin_amdgcn_perm(kHi, kLo, s0);
    d1 = __builtin_amdgcn_perm(kHi, kLo, s1);
}
__device__ __forceinline__ void field_to_bf16(uint32_t f, uint32_t &d0, uint32_t &d1) {
    // u = 0, 1, 2 -> low byte 0x80, 0x00, 0x80, high byte 0xBF, 0x00, 0x3F
    field_to_16<0x00800080u, 0x003F00BFu>(f, d0, d1);
}
__device__ __forceinline__ void field_to_half(uint32_t f, uint32_t &d0, uint32_t &d1) {
    field_to_16<0u, 0x003C00BCu>(f, d0, d1);  // -1 / 0 / +1 are 0xBC00 / 0x0000 / 0x3C00
}

// Base-3 decode table entry for byte v: its five trits t_r = c_r + 1 (first
// code in the least significant trit) as one field per byte, bytes 0..4.
// Bytes 243..255 are not produced by the packing; they read as five zero codes.
__device__ __forceinline__ uint64_t base3_field_entry(uint32_t v) {
    if (v >= 243u) return 0x0101010101ull;
    uint64_t e = 0;
#pragma unroll
    for (int r = 0; r < 5; ++r) {
        e |= (uint64_t)(v % 3u) << (8 * r);
        v /= 3u;
    }
    return e;
}

// Eight bytes of the base-3 layout (words w0, w1, first byte in the low bits)
// as their 40 fields, one per byte, looked up in the table; then the 32 fields
// starting at field `first` (0..4) as eight words of four fields each
// (natural order).
__device__ __forceinline__ void base3_fields(uint32_t w0, uint32_t w1, int first,
                                             const uint64_t *lut, uint32_t (&out)[8]) {
    uint64_t f[5] = {0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t v = ((i < 4 ? w0 : w1) >> (8 * (i % 4))) & 0xFFu;
        const uint64_t e = lut[v];
        constexpr int kSh[8] = {0, 40, 16, 56, 32, 8, 48, 24};  // 8 * (5 i % 8)
        const int w = (5 * i) / 8, sh = kSh[i];
        f[w] |= e << sh;
        if (sh > 24) f[w + 1] |= e >> (64 - sh);
    }
    const int sh = 8 * first;  // 0 .. 32
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const uint64_t lo = f[w] >> sh;
        const uint64_t hi = sh == 0 ? 0 : f[w + 1] << (64 - sh);
        const uint64_t v = lo | hi;
        out[2 * w] = (uint32_t)v;
        out[2 * w + 1] = (uint32_t)(v >> 32);
    }
}

// The same for 16 codes: four bytes hold the 16 fields from field `first` on.
__device__ __forceinline__ void base3_fields16(uint32_t w, int first, const uint64_t *lut,
                                               uint32_t (&out)[4]) {
    const uint64_t e0 = lut[w & 0xFFu], e1 = lut[(w >> 8) & 0xFFu], e2 = lut[(w >> 16) & 0xFFu],
                   e3 = lut[w >> 24];
    // bytes 0..4 of each entry, one after the other: five words
    const uint32_t f[5] = {(uint32_t)e0, (uint32_t)(e0 >> 32) | (uint32_t)e1 << 8,
                           (uint32_t)(e1 >> 24) | (uint32_t)e2 << 16,
                           (uint32_t)(e2 >> 16) | (uint32_t)e3 << 24, (uint32_t)(e3 >> 8)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        out[i] = first == 4 ? f[i + 1] : __builtin_amdgcn_alignbyte(f[i + 1], f[i], first);
}

// The top halves of two fp32 words as one word of two bf16 values.
__device__ __forceinline__ uint32_t top_halves(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// Piece `piece` of the exact three-way bf16 split of fp32 values x = hi + mid
// + lo: hi is x with its low 16 bits cleared, mid the same of x - hi, lo =
// x - hi - mid. Each subtraction is exact, and the pieces carry 8 + 8 + 8 of
// x's 24 significant bits, so every piece is a bf16 value (for |x| >= 2^-110;
// below that lo can fall among fp32 subnormals and lose bits under 2^-133).
// All pieces share x's sign, so |hi| + |mid| + |lo| = |x|.
__device__ __forceinline__ uint32_t f32_piece_bits(uint32_t ux, int piece) {
    if (piece == 0) return ux;
    const float x = __uint_as_float(ux);
    const float r = x - __uint_as_float(ux & 0xFFFF0000u);
    const uint32_t ur = __float_as_uint(r);
    if (piece == 1) return ur;
    return __float_as_uint(r - __uint_as_float(ur & 0xFFFF0000u));
}

}  // namespace
}  // namespace bl
