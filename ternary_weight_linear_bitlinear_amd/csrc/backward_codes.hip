// Backward products of a layer whose forward pass left INT8 codes, and of a stack
// of matrices that share their input, with the straight-through estimator ([QAT-en]
// "How Gradients Flow: Fake Quantization and STE"; [b158] §5.3):
//
//   grad_w[n, k] = sum_m v[m, n] * xq[m, k],  v = grad_y[m, n] * (scale[m] / 127)
//   grad_x[m, k] = sum_s gamma_s sum_{n in s} grad_y[m, n] * c[n, k]
//
// C[i, j] = sum_p A(i, p) B(p, j) on the bf16 matrix cores (v_mfma_f32_32x32x16_bf16)
// with fp32 sums, B stored [p][j]:
//   grad_w: i = n, j = k, p = m; A = v, read as [p][i]; B = the INT8 codes, exact in
//           bf16.
//   grad_x: i = m, j = k, p = n; A = grad_y as stored ([i][p]); B = packed codes,
//           expanded to bf16.
// An fp32 value of A (v is one: one rounding of its product) enters in pieces that the
// same fragment of B is multiplied by one after the other. Two ways:
//   three bf16 pieces of 8 significant bits each: exact, whatever the values. grad_w in
//   bf16 takes two of them (v to within 2^-15, far below its own rounding of 2^-8).
//   two fp16 pieces of 11 bits, rounded to nearest, for two thirds of the matrix-core work
//   (one for grad_w in bf16). fp16's range is short, so each row of C's values of A are
//   scaled by a power of two that brings the largest to 2^14 .. 2^15, and the result back.
//   A scaled value x is then off by 2^-22 x or 2^-25, whichever is more (one piece: 2^-11 x
//   or 2^-25). A first kernel finds each row's largest value and the least that is not
//   zero, and a tile takes fp16 only where no value of its rows can be off by more than
//   max(4, P) 2^-24 of itself, what a sum of P terms in fp32 may be off by anyway (one
//   piece: 2^-11). Other tiles take the bf16 pieces: beside a value 2^30 times theirs, whose
//   code is zero, the rest of a row would keep eight bits.
// Large tiles, bound by the matrix cores, take fp16 (weight gradient 4096^3 to fp32: 239 us
// and 9 us for the search; where the values of every tile lie too far apart 327 us in all);
// small ones, bound by
// latency, bf16 in one launch less (fp16 in them: 100 x 1003 x 2001 9.6 -> 11.7 us, 200 tokens
// over 2003 rows of 3000 29.6 -> 32.6 us).
//
// Each segment's sum has a factor of its own. Instead of a second set of sums the
// running sums are rescaled where a segment ends, by the ratio of its gamma to the
// next one's. The segments are taken in the order of |gamma|, so that a ratio is at
// most 1 and nothing overflows (0 / 0: every sum so far counts for nothing and the
// ratio is 1); the last one's gamma multiplies the result.
//
// The operands go through LDS in their natural layout, two stages of it; fragments
// whose contraction index runs along LDS rows are read with the transposing load,
// as in backward.hip.
//
// What bounds it: large tiles keep the matrix cores busy for 57-60% of a compute unit's
// cycles at the clock that their power leaves (weight gradient 4096^3: 2 x 137 GFLOP in 239 us,
// 1.15 PFLOP/s; input gradient of 2048 tokens over 2 x 11008 rows of 4096: 369 GFLOP in 297
// us, 1.24 PFLOP/s; a library product of 8192^3 in bf16 reaches 1.2). Unaligned rows cost the
// weight gradient 6 to 19%, the input gradient from fp32 20% and from bf16 19 (1-bit) to 54%
// (2-bit, base-3): ends that load element by element, branches behind the loads, and 4 to 11
// spilled registers in its large tiles. Small tiles wait: of a
// stage's 0.8 us (fp32, three pieces, aligned) 0.2 are loads and their addresses, 0.2 the
// conversion, and the matrix cores' third hides behind the rest. Tried there and not
// kept: loads two stages ahead (the same times), a stage's fragments read at once (29.5 -> 31.8 us),
// half as long slices and twice the workgroups (27 -> 31 us for 300 tokens over 2 x 2000 rows).
#include "backward_util.hpp"
#include "bl_internal.hpp"
#include "device_util.hpp"
#include "row_share.hpp"

#include <cmath>

namespace bl {
namespace {

constexpr int kXcds = 8;
enum { kBCodes8 = 0, kBPacked2 = 1, kBPacked1 = 2, kBPacked3 = 3 };

struct CodesArgs {
    const void *A;
    int64_t lda;
    const void *B;
    int64_t ldb;
    const float *scale;  // grad_w: the tokens' scales
    GammaMap gm;         // grad_x: the segments
    int64_t I, J, P;
    int tiles_i, tiles_j;
    int splits;   // workgroups that share a tile's slices
    const uint2 *peak;  // fp16 pieces: the largest |A(i, .)| (a float's bits) and the least
                        // that is not zero (its least_key), [peaks, I]
    int peaks;
    void *C;      // [I, J]; with splits their partial sums, [splits, I, J] fp32
    float floor;  // what the least one has to be where the largest is 2^14 .. 2^15
};

// Block tile BI x BJ outputs, contraction slice BP per stage, WI x WJ waves.
template <int BI_, int BJ_, int BP_, int WI_, int WJ_>
struct Tile {
    static constexpr int BI = BI_, BJ = BJ_, BP = BP_, WI = WI_, WJ = WJ_;
    static constexpr int kThreads = 64 * WI * WJ;
    static constexpr int FI = BI / WI / 32, FJ = BJ / WJ / 32;
    static constexpr int KSTEPS = BP / 16;
};
// What a stage of NP pieces of A and one B takes in LDS. Padded rows: of an [i][p]
// tile by 16 bytes, which puts 16 rows of 16-byte reads on distinct banks; of [p][*]
// tiles by 64, which keeps the four rows of a transposing load apart; B's short rows by
// 32, which does too, so that two workgroups with base-3's table fit a compute unit
// (200 x 2003 x 3000 from fp32: 45 -> 29 us).
template <typename T, bool A_T, int BSRC, int NP>
struct Stage {
    static constexpr int LD_A = A_T ? T::BI * 2 + 64 : T::BP * 2 + 16;
    static constexpr int LD_B = T::BJ * 2 + (T::BJ == 64 ? 32 : 64);
    static constexpr int PLANE = A_T ? T::BP * LD_A : T::BI * LD_A;  // one piece of A
    static constexpr int BYTES = NP * PLANE + T::BP * LD_B;
    static constexpr int LUT = BSRC == kBPacked3 ? 256 * 8 : 0;
    static constexpr int SMEM = 2 * BYTES + LUT;
    static_assert(SMEM <= (int)kLdsBytesPerCu, "two stages in LDS");
};

// LDS slot of 16-byte piece `c` of row `row` of B. A thread writes its codes' pieces
// (two or four) one after the other, so that the lanes of one write stand 32 or 64
// bytes apart and would meet on a quarter or a half of the banks; the pieces of a
// thread are permuted so that lanes and neighbouring rows take different ones (input
// gradient, 4096^3: a third of the LDS cycles were conflicts). Rows r and r + 4 have
// the same order, so that a transposing load's lanes keep one offset.
template <int BSRC>
__device__ __forceinline__ int b_slot(int row, int c) {
    if constexpr (BSRC == kBCodes8) return c ^ (c / 16 & 1);
    const int u = c / 4;
    return c ^ ((u + u / 4 + 3 * row) & 3);
}

// Eight elements from any address; those from `count` on are zero and not read.
template <typename T>
__device__ __forceinline__ void load8_some(const T *p, int64_t count, Raw8<T> &r) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < count ? Elem<T>::get(p, e) : 0.f;
    if constexpr (sizeof(T) == 4) {
        r.a = make_float4(v[0], v[1], v[2], v[3]);
        r.b = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = top_halves(__float_as_uint(v[2 * e]), __float_as_uint(v[2 * e + 1]));
        r.a = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
// Two values as two fp16 ones, rounded to nearest, in a word.
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ half2_t to_half2(float a, float b) {
    return __builtin_convertvector(float2_t{a, b}, half2_t);
}
// The power of two that takes a row's largest value to 2^14 .. 2^15 (any, for rows of
// values below 2^-112), and its inverse.
__device__ __forceinline__ float peak_scale(float top) {
    uint32_t e = __float_as_uint(top) >> 23;
    e = e < 15u ? 15u : e;
    return __uint_as_float((268u - e) << 23);
}
__device__ __forceinline__ float power_inverse(float scale) {
    return __uint_as_float((254u << 23) - __float_as_uint(scale));
}
// The order of |v| with zeros last: its bits without the sign, doubled, less one.
__device__ __forceinline__ uint32_t least_key(float v) { return 2u * __float_as_uint(v) - 1u; }
constexpr uint32_t kNoLeast = 0xFFFFFFFFu;
__device__ __forceinline__ float least_of(uint32_t key) { return __uint_as_float((key + 1u) / 2u); }

// Memory of `bytes` bytes (as many as 32 bits hold) from a uniform address, as buffer
// loads take it: offsets past it read zeros.
typedef int v2i __attribute__((ext_vector_type(2)));
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, int64_t bytes) {
    const uint32_t n = bytes < 0xFFFFFFFFll ? (uint32_t)bytes : 0xFFFFFFFFu;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)n, 0x00020000);
}
__device__ __forceinline__ v4i load_v4(__amdgpu_buffer_rsrc_t b, uint32_t at) {
    return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(b, (int)at, 0, 0));
}
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)v) |
                     (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32);
}

// x / 127, correctly rounded (Markstein's step from the rounded reciprocal).
__device__ __forceinline__ float over127(float x) {
    constexpr float r = 1.0f / 127.0f;
    const float q = x * r;
    return __builtin_fmaf(__builtin_fmaf(-127.0f, q, x), r, q);
}

// VEC: A's rows and segments begin at multiples of 8 elements, xq's at multiples of
// 16 (aligned loads).
//
// A stage's loads go to registers while the stage before it is multiplied, and from
// there, converted, to LDS between the matrix-core instructions of that same stage:
// the vector unit's work then runs in their shadow, and the registers are free for
// the loads of the next stage at once. Fragments are read one group of
// instructions ahead.
template <typename T, bool A_T, int BSRC, int NP, bool HALF, bool VEC, typename GT, typename OT>
__device__ __forceinline__ bool codes_gemm_tile(const CodesArgs a) {
    using S = Stage<T, A_T, BSRC, NP>;
    constexpr int kT = T::kThreads;
    static_assert(A_T == (BSRC == kBCodes8), "grad_w from INT8 codes, grad_x from packed ones");
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint64_t *lut = reinterpret_cast<uint64_t *>(smem + 2 * S::BYTES);  // base-3 only

    const int ntiles = a.tiles_i * a.tiles_j;
    const int per_xcd = (ntiles * a.splits + kXcds - 1) / kXcds;
    int t = (blockIdx.x % kXcds) * per_xcd + blockIdx.x / kXcds;
    if (t >= ntiles * a.splits) return true;
    const int split = t / ntiles;
    t -= split * ntiles;
    const int64_t i0 = (int64_t)(t / a.tiles_j) * T::BI;
    const int64_t j0 = (int64_t)(t % a.tiles_j) * T::BJ;
    const int tid = threadIdx.x;
    const int wave = tid / 64, lane = tid % 64;
    const int wi = wave / T::WJ, wj = wave % T::WJ;

    // Segments in the order of |gamma|: where they begin and end, and the factor
    // that the sums take before the segment's own terms.
    __shared__ int64_t seg_begin[kMaxSegments], seg_end[kMaxSegments];
    __shared__ float seg_ratio[kMaxSegments], seg_gamma[kMaxSegments];
    const int nseg = A_T ? 1 : a.gm.nseg;
    if constexpr (!A_T) {
        if (tid < nseg) {
            // (magnitudes compared as integers, which is an order of every gamma, NaN
            // too: each segment has a rank of its own)
            const float mine = a.gm.g[tid];
            auto size = [](float g) { return __float_as_uint(g) & 0x7FFFFFFFu; };
            int rank = 0;
            float before = 0.f;  // of the largest |gamma| that goes before
            for (int s = 0; s < nseg; ++s) {
                const float g = a.gm.g[s];
                if (size(g) < size(mine) || (size(g) == size(mine) && s < tid)) {
                    ++rank;
                    if (size(g) >= size(before)) before = g;
                }
            }
            seg_begin[rank] = tid == 0 ? 0 : a.gm.bound[tid - 1];
            seg_end[rank] = tid == nseg - 1 ? a.P : a.gm.bound[tid];
            seg_ratio[rank] = mine == 0.f ? 1.0f : before / mine;
            seg_gamma[rank] = mine;
        }
        if constexpr (BSRC == kBPacked3) {
            for (int i = tid; i < 256; i += kT) lut[i] = base3_field_entry((uint32_t)i);
        }
        __syncthreads();
    }

    // ---- global -> registers ------------------------------------------------------
    constexpr int A_ROW = A_T ? T::BI / 8 : T::BP / 8;  // chunks of eight in a tile row
    constexpr int A_CH = T::BI * T::BP / 8 / kT;
    static_assert(A_CH * 8 * kT == T::BI * T::BP && kT % A_ROW == 0, "whole chunks for every thread");
    constexpr int A_STEP = kT / A_ROW;  // tile rows between a thread's chunks
    // codes for each thread: 32 packed ones where that leaves none idle; threads of a row
    constexpr int B_EACH = BSRC != kBCodes8 && T::BP * T::BJ / 32 >= kT ? 32 : 16, B_ROW = T::BJ / B_EACH;
    constexpr int B_CH = (T::BP * B_ROW + kT - 1) / kT;
    static_assert(T::BP * B_ROW % kT == 0 || T::BP * B_ROW < kT, "whole rows of B");
    constexpr int B_STEP = kT / B_ROW;
    Raw8<GT> a_reg[A_CH];
    float a_scale[A_T ? A_CH : 1];
    v4i b_reg[B_CH];  // grad_w: 16 codes of one token; packed: as unpacked below
    const int ar = tid / A_ROW, ac = tid % A_ROW;
    const int br = tid / B_ROW, bc = tid % B_ROW;
    const bool b_mine = T::BP * B_ROW >= kT || br < T::BP;
    const GT *const A = static_cast<const GT *>(a.A);
    const uint8_t *const B = static_cast<const uint8_t *>(a.B);

    // Where the thread's pieces lie, in bytes from a uniform address (at most 127 rows
    // on: the limits of the calls keep that below 2^32). Rows of an [i][p] tile past I
    // read the last one, columns past the matrix the tile's first: they only reach
    // outputs that are not stored.
    uint32_t a_off[A_CH];
    const GT *a_base[A_T ? 1 : A_CH];
    if constexpr (A_T) {
        a_base[0] = A + i0;
        a_off[0] = (uint32_t)((ar * a.lda + (i0 + 8 * ac < a.I ? 8 * ac : 0)) * sizeof(GT));
    } else {
#pragma unroll
        for (int c = 0; c < A_CH; ++c) {
            const int64_t first = i0 + c * A_STEP < a.I ? i0 + c * A_STEP : a.I - 1;
            a_base[c] = A + first * a.lda;
            a_off[c] = (uint32_t)(((first + ar < a.I ? ar : a.I - 1 - first) * a.lda + 8 * ac) * sizeof(GT));
        }
    }
    const int64_t c0 = j0 + (int64_t)B_EACH * bc;  // B's columns
    constexpr int kPer = BSRC == kBCodes8 ? 1 : BSRC == kBPacked2 ? 4 : BSRC == kBPacked1 ? 8 : 5;
    // (packed rows are whole 16-byte pieces; dwords past a row are taken from its start)
    const int64_t b_first = c0 / kPer & ~(int64_t)3;
    // the dwords that hold the codes (base-3 rows: from any byte on)
    constexpr int kWords = BSRC == kBPacked2 ? B_EACH / 16 : BSRC == kBPacked1 ? 1 : B_EACH / 16 + 1;
    int b_at[3];  // bytes from the row's start; codes: the first only
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int64_t at = b_first + 4 * i;
        b_at[i] = BSRC == kBCodes8 ? (c0 < a.J ? (int)c0 : 0) : at < a.ldb ? (int)at : 0;
    }
    const int b_shift = BSRC == kBPacked3 ? (int)(c0 / 5 - b_first) : BSRC == kBPacked1 ? (int)(c0 % 32 / 4) : 0;
    const int b_code = BSRC == kBPacked3 ? (int)(c0 % 5) : 0;

    // fp16 pieces: the powers of two of the thread's columns (A_T) or rows, inverses for the
    // end; and whether every row's values are near enough to its largest for them.
    __shared__ float inverse[HALF ? T::BI : 1];
    __shared__ int apart;
    float a_pow[HALF ? (A_T ? 8 : A_CH) : 1];
    if constexpr (HALF) {
        // (over the runs: every thread takes a row's share)
        constexpr int kShares = kT / T::BI;
        static_assert(kShares >= 1 && kT % T::BI == 0, "a thread for each row of the tile");
        float *red = reinterpret_cast<float *>(smem);  // [kShares][BI]
        const int col = tid % T::BI, share = tid / T::BI;
        const int64_t i = i0 + col < a.I ? i0 + col : a.I - 1;
        float top = 0.f;
        uint32_t least = kNoLeast;
#pragma unroll 8
        for (int n = share; n < a.peaks; n += kShares) {
            const uint2 v = a.peak[n * a.I + i];
            top = fmaxf(top, __uint_as_float(v.x));
            least = min(least, v.y);
        }
        red[tid] = top;
        if (tid == 0) apart = 0;
        __syncthreads();
        auto scale_of = [&](int row) {
            float t = red[row];
#pragma unroll
            for (int n = 1; n < kShares; ++n) t = fmaxf(t, red[n * T::BI + row]);
            return peak_scale(t);
        };
#pragma unroll
        for (int e = 0; e < (A_T ? 8 : A_CH); ++e) a_pow[e] = scale_of(A_T ? 8 * ac + e : ar + e * A_STEP);
        const float scale = scale_of(col);
        if (tid < T::BI) inverse[tid] = power_inverse(scale);
        if (least != kNoLeast && !(least_of(least) * scale >= a.floor)) apart = 1;
        __syncthreads();  // the memory is the stages' from here on
        if (__builtin_amdgcn_readfirstlane(apart)) return false;
    }

    // Aligned rows load from buffers that end with the segment: what lies past it reads
    // as zero (A needs that; a token's scale of zero does the same for its row), and no
    // load has a branch or a select behind it. Of an [i][p] tile the columns past a
    // segment's end are sent past the buffer's. (Unaligned fp32 rows of it load the
    // same way, from a buffer that ends with the matrix; store_a clears their ends.)
    const uint32_t b_row = (uint32_t)(br * a.ldb);
    auto load_a_vec = [&](int c, int64_t p0, int64_t p1) __attribute__((always_inline)) {
        const GT *at = A_T ? a_base[0] + p0 * a.lda : a_base[A_T ? 0 : c] + p0;
        uint32_t off = a_off[A_T ? 0 : c];
        if constexpr (A_T) off += (uint32_t)(c * A_STEP * a.lda * sizeof(GT));
        else if constexpr (VEC) off = p0 + 8 * ac < p1 ? off : 0xFFFFFFFFu;
        const auto buf = buffer_of(at, A_T ? ((p1 - p0) * a.lda - i0) * (int64_t)sizeof(GT)
                                           : VEC ? 0xFFFFFFF0ll : (A + a.I * a.lda - at) * (int64_t)sizeof(GT));
        const v4i q = load_v4(buf, off);
        if constexpr (sizeof(GT) == 2) {
            a_reg[c].a = __builtin_bit_cast(uint4, q);
        } else {
            a_reg[c].a = __builtin_bit_cast(float4, q);
            a_reg[c].b = __builtin_bit_cast(float4, load_v4(buf, VEC && !A_T ? off | 16 : off + 16));
        }
        if constexpr (A_T)
            a_scale[c] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                buffer_of(a.scale + p0, (p1 - p0) * 4), 4 * (ar + c * A_STEP), 0, 0));
    };
    auto load_b_vec = [&](int c, int64_t p0, int64_t p1) __attribute__((always_inline)) {
        const auto buf = buffer_of(B + p0 * a.ldb, (p1 - p0) * a.ldb);
        const uint32_t row = b_row + (uint32_t)(c * B_STEP * a.ldb);
        if constexpr (BSRC == kBCodes8) {
            b_reg[c] = load_v4(buf, row + b_at[0]);
        } else if constexpr (BSRC == kBPacked2 && B_EACH == 32) {
            const v2i v = __builtin_bit_cast(v2i, __builtin_amdgcn_raw_buffer_load_b64(buf, row + b_at[0], 0, 0));
            b_reg[c] = v4i{v[0], v[1], 0, 0};
        } else {
            int d[3] = {0, 0, 0};
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                d[i] = __builtin_bit_cast(int, __builtin_amdgcn_raw_buffer_load_b32(buf, row + b_at[i], 0, 0));
            b_reg[c] = v4i{d[0], d[1], d[2], 0};
        }
    };
    // Other rows load unaligned pieces, which run on past a row's or a segment's end into
    // what follows; where too little does, at the end of the matrix, element by element.
    // (Behind a piece of a [p][i] tile up to 15 elements: 16 rows hold them at least.
    // Behind one of an [i][p] tile up to BP: the rows after the tile's have to.)
    auto load_a_any = [&](int c, int64_t p0, int64_t p1) __attribute__((always_inline)) {
        const int row = ar + c * A_STEP;
        if constexpr (A_T) {
            const int64_t p = p0 + row < p1 ? p0 + row : p1 - 1;
            a_scale[c] = p0 + row < p1 ? a.scale[p] : 0.f;
            if (i0 + T::BI <= a.I || p0 + T::BP + 16 <= p1) {
                load_any(a_base[0] + p * a.lda + (i0 + 8 * ac < a.I ? 8 * ac : 0), a_reg[c]);
            } else {
                const int64_t i = i0 + 8 * ac;
                load8_some(A + p * a.lda + (i < a.I ? i : 0), i < a.I ? a.I - i : 0, a_reg[c]);
            }
        } else if (p0 + T::BP <= a.lda || (a.I - i0 - T::BI) * a.lda >= T::BP) {
            const GT *at = a_base[A_T ? 0 : c] + p0;
            load_any(reinterpret_cast<const GT *>(reinterpret_cast<const char *>(at) + a_off[c]), a_reg[c]);
        } else {
            const int64_t i = i0 + row, p = p0 + 8 * ac;
            const bool ok = i < a.I && p < p1;
            load8_some(A + (ok ? i * a.lda + p : 0), ok ? p1 - p : 0, a_reg[c]);
        }
    };
    auto load_b_any = [&](int c, int64_t p0, int64_t p1) __attribute__((always_inline)) {
        if constexpr (BSRC == kBCodes8) {
            const int64_t p = p0 + br + c * B_STEP;
            const uint8_t *row = B + (p < p1 ? p : p1 - 1) * a.ldb;
            if (j0 + T::BJ <= a.J || p0 + T::BP + 16 <= p1) {
                b_reg[c] = load16_any(reinterpret_cast<const int8_t *>(row) + b_at[0]);
                return;
            }
            uint32_t d[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (c0 + e < a.J) d[e / 4] |= (uint32_t)row[c0 + e] << (8 * (e % 4));
            b_reg[c] = v4i{(int)d[0], (int)d[1], (int)d[2], (int)d[3]};
        } else {
            load_b_vec(c, p0, p1);  // (packed rows are aligned whatever K is)
        }
    };
    auto load_a = [&](int c, int64_t p0, int64_t p1) __attribute__((always_inline)) {
        if constexpr (VEC || (!A_T && sizeof(GT) == 4)) load_a_vec(c, p0, p1);
        else load_a_any(c, p0, p1);
    };
    auto load_b = [&](int c, int64_t p0, int64_t p1) __attribute__((always_inline)) {
        if constexpr (VEC) load_b_vec(c, p0, p1);
        else if (b_mine) load_b_any(c, p0, p1);
    };

    // ---- registers -> LDS -----------------------------------------------------------
    // (rest: contraction indexes from the slice's first to the segment's end)
    auto store_a = [&](uint8_t *st, int c, int64_t rest) __attribute__((always_inline)) {
        uint8_t *dst = st + (ar + c * A_STEP) * S::LD_A + 16 * ac;
        const bool ends = !VEC && !A_T && rest < T::BP;  // uniform
        if constexpr (NP == 1 && !HALF) {
            v4i w = __builtin_bit_cast(v4i, a_reg[c].a);
            if (ends) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] &= (8 * ac + 2 * e < rest ? 0xFFFF : 0) | (8 * ac + 2 * e + 1 < rest ? (int)0xFFFF0000u : 0);
            }
            *reinterpret_cast<v4i *>(dst) = w;
        } else {
            float v[8];
            a_reg[c].widen(v);
            if (ends) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = 8 * ac + e < rest ? v[e] : 0.f;
            }
            if constexpr (A_T) {
                const float f = over127(a_scale[c]);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= f;
            }
            if constexpr (HALF) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= a_pow[A_T ? e : c];
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    v4i w;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const half2_t h = to_half2(v[2 * e], v[2 * e + 1]);
                        w[e] = __builtin_bit_cast(int, h);
                        v[2 * e] -= (float)h[0];
                        v[2 * e + 1] -= (float)h[1];
                    }
                    *reinterpret_cast<v4i *>(dst + n * S::PLANE) = w;
                }
                return;
            }
#pragma unroll
            for (int n = 0; n < NP; ++n) {  // each piece of what the ones before leave
                v4i w;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = (int)top_halves(__float_as_uint(v[2 * e]), __float_as_uint(v[2 * e + 1]));
                *reinterpret_cast<v4i *>(dst + n * S::PLANE) = w;
                if (n + 1 < NP) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] -= __uint_as_float(__float_as_uint(v[e]) & 0xFFFF0000u);
                }
            }
        }
    };
    auto store_b = [&](uint8_t *st, int c) __attribute__((always_inline)) {
        if (!b_mine) return;
        const int row = br + c * B_STEP;
        uint8_t *dst = st + NP * S::PLANE + row * S::LD_B;
        uint32_t d[B_EACH / 2];
        auto field = [](uint32_t f, uint32_t &d0, uint32_t &d1) {
            if constexpr (HALF) field_to_half(f, d0, d1);
            else field_to_bf16(f, d0, d1);
        };
        if constexpr (BSRC == kBCodes8) {
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const uint32_t w = (uint32_t)b_reg[c][e / 4];
                const float lo = (float)(int8_t)(w >> (8 * (e % 4))), hi = (float)(int8_t)(w >> (8 * (e % 4 + 1)));
                d[e / 2] = HALF ? __builtin_bit_cast(uint32_t, to_half2(lo, hi))
                                : top_halves(__float_as_uint(lo), __float_as_uint(hi));
            }
        } else if constexpr (BSRC == kBPacked1) {
            // bit t of byte i is code 4 t + i; u = 2 bit picks -1 or +1
            const uint32_t w = (uint32_t)b_reg[c][0] >> b_shift;
#pragma unroll
            for (int t = 0; t < B_EACH / 4; ++t) field(((w >> t) & 0x01010101u) << 1, d[2 * t], d[2 * t + 1]);
        } else if constexpr (BSRC == kBPacked3) {
            // the four or eight bytes of the codes lie in one dword more
            uint32_t f[B_EACH / 4];
            const uint32_t lo = __builtin_amdgcn_alignbyte(b_reg[c][1], b_reg[c][0], b_shift);
            if constexpr (B_EACH == 16)
                base3_fields16(lo, b_code, lut, f);
            else
                base3_fields(lo, __builtin_amdgcn_alignbyte(b_reg[c][2], b_reg[c][1], b_shift), b_code, lut, f);
#pragma unroll
            for (int w = 0; w < B_EACH / 4; ++w) field(f[w], d[2 * w], d[2 * w + 1]);
        } else {
            // field s of a word holds its codes 4 s .. 4 s + 3
#pragma unroll
            for (int w = 0; w < B_EACH / 16; ++w)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    field(((uint32_t)b_reg[c][w] >> (2 * s)) & 0x03030303u, d[8 * w + 2 * s],
                                  d[8 * w + 2 * s + 1]);
        }
#pragma unroll
        for (int q = 0; q < B_EACH / 8; ++q)
            *reinterpret_cast<uint4 *>(dst + 16 * b_slot<BSRC>(row, B_EACH / 8 * bc + q)) =
                make_uint4(d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]);
    };

    // ---- fragments --------------------------------------------------------------------
    const int g16 = lane / 16, t16 = lane % 16;
    auto tr_frag = [&](const uint8_t *p, int ld) __attribute__((always_inline)) -> bf16x8 {
        const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p));
        const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p + 4 * ld));
        const v8s both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf16x8, both);
    };
    const int tr_row = 8 * (g16 / 2) + t16 / 4, tr_col = 2 * (16 * (g16 % 2) + 4 * (t16 % 4));
    const int a_lane = A_T ? tr_row * S::LD_A + tr_col + wi * (T::BI / T::WI) * 2
                           : (wi * (T::BI / T::WI) + lane % 32) * S::LD_A + 16 * (lane / 32);
    int b_lane[T::FJ];
#pragma unroll
    for (int j = 0; j < T::FJ; ++j) {
        const int col = tr_col + (wj * (T::BJ / T::WJ) + 32 * j) * 2;  // bytes
        b_lane[j] = NP * S::PLANE + tr_row * S::LD_B + 16 * b_slot<BSRC>(tr_row, col / 16) + col % 16;
    }
    auto a_frag = [&](const uint8_t *st, int ks, int n, int i) __attribute__((always_inline)) -> bf16x8 {
        const uint8_t *p = st + a_lane + n * S::PLANE;
        if constexpr (A_T) return tr_frag(p + 16 * ks * S::LD_A + i * 64, S::LD_A);
        else return *reinterpret_cast<const bf16x8 *>(p + i * 32 * S::LD_A + 32 * ks);
    };
    auto b_frag = [&](const uint8_t *st, int ks, int j) __attribute__((always_inline)) -> bf16x8 {
        return tr_frag(st + b_lane[j] + 16 * ks * S::LD_B, S::LD_B);
    };
    v16f acc[T::FI][T::FJ];
#pragma unroll
    for (int i = 0; i < T::FI; ++i)
#pragma unroll
        for (int j = 0; j < T::FJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    // ---- the slices of every segment in turn --------------------------------------------
    struct Slice {
        int seg;
        int64_t p, end;
    };
    auto begin_of = [&](int s) { return A_T ? (int64_t)0 : uniform(seg_begin[s]); };
    auto end_of = [&](int s) { return A_T ? a.P : uniform(seg_end[s]); };
    auto after = [&](Slice s) {  // the last one again past the end
        if (s.p + T::BP < s.end) {
            s.p += T::BP;
        } else if (s.seg + 1 < nseg) {
            ++s.seg;
            s.p = begin_of(s.seg), s.end = end_of(s.seg);
        }
        return s;
    };
    // this workgroup's share of them: `left` slices from cur on
    int64_t slices = 0;
    for (int s = 0; s < nseg; ++s) slices += (end_of(s) - begin_of(s) + T::BP - 1) / T::BP;
    int64_t skip = slices * split / a.splits, left = slices * (split + 1) / a.splits - skip;
    Slice cur{0, begin_of(0), end_of(0)};
    for (int64_t n; skip >= (n = (cur.end - cur.p + T::BP - 1) / T::BP);) {
        skip -= n;
        ++cur.seg;
        cur.p = begin_of(cur.seg);
        cur.end = end_of(cur.seg);
    }
    cur.p += skip * T::BP;
    // Registers hold the next slice, LDS the current one. A piece's register is loaded
    // again as soon as it has been converted, so that every load has a whole stage's
    // time; past the last slice it is loaded and converted again, and never multiplied.
    // (Unaligned rows, whose ends may load element by element, leave that out.)
    constexpr int kTasks = A_CH + B_CH;
    auto task = [&](int q, uint8_t *to, const Slice &held, const Slice &s, bool real) __attribute__((always_inline)) {
        if (q < A_CH) {
            store_a(to, q, held.end - held.p);
            if (VEC || real) load_a(q, s.p, s.end);
        } else {
            store_b(to, q - A_CH);
            if (VEC || real) load_b(q - A_CH, s.p, s.end);
        }
    };
#pragma unroll
    for (int c = 0; c < A_CH; ++c) load_a(c, cur.p, cur.end);
#pragma unroll
    for (int c = 0; c < B_CH; ++c) load_b(c, cur.p, cur.end);
    Slice next = after(cur);
#pragma unroll
    for (int q = 0; q < kTasks; ++q) task(q, smem, cur, next, left > 1);
    __syncthreads();
    // A stage's groups of instructions: one piece of A and one k-step each, their
    // fragments read a group ahead.
    constexpr int kGroups = T::KSTEPS * NP;
    bf16x8 af[2][T::FI], bb[2][T::FJ];
    auto read_frags = [&](const uint8_t *st, int g) __attribute__((always_inline)) {
        const int ks = g / NP, n = g % NP;
        if (n == 0) {
#pragma unroll
            for (int j = 0; j < T::FJ; ++j) bb[ks & 1][j] = b_frag(st, ks, j);
        }
#pragma unroll
        for (int i = 0; i < T::FI; ++i) af[g & 1][i] = a_frag(st, ks, n, i);
    };
    auto multiply = [&](int g) __attribute__((always_inline)) {
        const int ks = g / NP;
#pragma unroll
        for (int i = 0; i < T::FI; ++i)
#pragma unroll
            for (int j = 0; j < T::FJ; ++j) {
                if constexpr (HALF)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                        __builtin_bit_cast(half8_t, af[g & 1][i]), __builtin_bit_cast(half8_t, bb[ks & 1][j]),
                        acc[i][j], 0, 0, 0);
                else
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[g & 1][i], bb[ks & 1][j],
                                                                        acc[i][j], 0, 0, 0);
            }
    };
    for (int buf = 0;; buf ^= 1) {
        const uint8_t *st = smem + buf * S::BYTES;
        uint8_t *to = smem + (buf ^ 1) * S::BYTES;
        const Slice then = after(next);
        read_frags(st, 0);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            if (g + 1 < kGroups) read_frags(st, g + 1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(g);
            // this group's share of the next stage
#pragma unroll
            for (int q = g * kTasks / kGroups; q < (g + 1) * kTasks / kGroups; ++q) task(q, to, next, then, left > 2);
        }
        if (left == 1) break;
        if (!A_T && next.seg != cur.seg) {  // (grad_w has one segment)
            const float f = seg_ratio[next.seg];
#pragma unroll
            for (int i = 0; i < T::FI; ++i)
#pragma unroll
                for (int j = 0; j < T::FJ; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[i][j][r] *= f;
        }
        cur = next;
        next = then;
        --left;
        lds_barrier();
    }

    // ---- epilogue: lane holds D[i][j] for j = lane % 32 and
    // i = 8 (r / 4) + 4 (lane / 32) + r % 4, register r
    const float alpha = A_T ? 1.0f : seg_gamma[cur.seg];
    OT *C = static_cast<OT *>(a.C) + split * a.I * a.J;
#pragma unroll
    for (int fi = 0; fi < T::FI; ++fi)
#pragma unroll
        for (int fj = 0; fj < T::FJ; ++fj) {
            const int64_t j = j0 + wj * (T::BJ / T::WJ) + fj * 32 + lane % 32;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = wi * (T::BI / T::WI) + fi * 32 + 8 * (r / 4) + 4 * (lane / 32) + r % 4;
                float v = acc[fi][fj][r];
                // (the power of two first: with it still in, gamma could take a sum that fp32
                // holds past its range)
                if constexpr (HALF) v *= inverse[row];
                if constexpr (!A_T) v *= alpha;
                if (i0 + row < a.I && j < a.J) put(C, (i0 + row) * a.J + j, v);
            }
        }
    return true;
}

// HALF: NP fp16 pieces, or EXACT bf16 ones in tiles whose rows' values lie too far apart
// (the tile gives up before its first load). One kernel for both, as a second one whose tiles
// end at once would be a launch more for every call; the input gradient takes as long as with
// fp16 alone, the weight gradient 1 to 2 us more (300 x 4096 x 4096 36.0 -> 37.2 us).
template <typename T, bool A_T, int BSRC, int NP, bool HALF, int EXACT, bool VEC, typename GT, typename OT>
__global__ __launch_bounds__(T::kThreads) void codes_gemm_kernel(const CodesArgs a) {
    if (!codes_gemm_tile<T, A_T, BSRC, NP, HALF, VEC, GT, OT>(a))
        codes_gemm_tile<T, A_T, BSRC, EXACT, false, VEC, GT, OT>(a);
}

// The largest |v| of each column of grad_y [M, N] over a run of tokens and the least that
// is not zero: eight columns and every eighth token of the run for each thread.
template <typename GT, bool VEC>
__global__ __launch_bounds__(256) void codes_peak_cols_kernel(const GT *grad_y, const float *scale, int64_t M,
                                                              int64_t N, uint2 *peak) {
    __shared__ float red[8][256];
    __shared__ uint32_t low[8][256];
    const int r = threadIdx.x / 32;
    const int64_t n0 = (int64_t)blockIdx.x * 256;
    const int left = (int)(N - n0 < 256 ? N - n0 : 256);
    const Share<1, VEC> sh{left, (int)threadIdx.x % 32, 32};
    const int64_t m0 = M * blockIdx.y / gridDim.y, m1 = M * (blockIdx.y + 1) / gridDim.y;
    float top[8];
    uint32_t lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) top[e] = 0.f, lo[e] = kNoLeast;
    for (int64_t m = m0 + r; m < m1; m += 32) {
        RowRegs<GT, 1, VEC> g[4];
        float f[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {  // (tokens past the run read its last one)
            const int64_t mu = m + 8 * u < m1 ? m + 8 * u : m1 - 1;
            g[u].load(grad_y + mu * N + n0, sh);
            f[u] = over127(scale[mu]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float v[8];
            g[u].widen(0, sh, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] *= f[u];
                top[e] = fmaxf(top[e], fabsf(v[e]));
                lo[e] = min(lo[e], least_key(v[e]));
            }
        }
    }
    const int start = sh.start(0), skip = sh.skip(0);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e >= skip) red[r][start + e] = top[e], low[r][start + e] = lo[e];
    __syncthreads();
    if ((int)threadIdx.x >= left) return;
    float t = red[0][threadIdx.x];
    uint32_t l = low[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        t = fmaxf(t, red[i][threadIdx.x]);
        l = min(l, low[i][threadIdx.x]);
    }
    peak[blockIdx.y * N + n0 + threadIdx.x] = make_uint2(__float_as_uint(t), l);
}
// The same of each row of grad_y (fp32): a workgroup for every row, or every gridDim.x-th.
__global__ __launch_bounds__(256) void codes_peak_rows_kernel(const float *grad_y, int64_t M, int64_t N,
                                                              uint2 *peak) {
    __shared__ float red[4];
    __shared__ uint32_t low[4];
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        const float *row = grad_y + m * N;
        float top = 0.f;
        uint32_t lo = kNoLeast;
        auto take = [&](float v) {
            top = fmaxf(top, fabsf(v));
            lo = min(lo, least_key(v));
        };
        if (N % 4 == 0) {
            for (int64_t n = (int64_t)threadIdx.x * 4; n < N; n += 1024) {
                const float4 v = *reinterpret_cast<const float4 *>(row + n);
                take(v.x), take(v.y), take(v.z), take(v.w);
            }
        } else {
            for (int64_t n = threadIdx.x; n < N; n += 256) take(row[n]);
        }
        top = wave_max0_dpp(top);
#pragma unroll
        for (int o = 32; o > 0; o /= 2) lo = min(lo, (uint32_t)__shfl_xor((int)lo, o, 64));
        if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = top, low[threadIdx.x / 64] = lo;
        __syncthreads();
        if (threadIdx.x == 0) {
            top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
            peak[m] = make_uint2(__float_as_uint(top), min(min(low[0], low[1]), min(low[2], low[3])));
        }
        __syncthreads();
    }
}

// out = the sum of `splits` partial results, in order.
template <typename OT>
__global__ __launch_bounds__(256) void codes_sum_kernel(const float *__restrict__ part, OT *__restrict__ out,
                                                        int64_t count, int splits) {
    const int64_t stride = (int64_t)gridDim.x * 256 * 4;
    int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (count % 4 == 0) {
        for (; at < count; at += stride) {
            float4 s = *reinterpret_cast<const float4 *>(part + at);
            for (int n = 1; n < splits; ++n) {
                const float4 q = *reinterpret_cast<const float4 *>(part + n * count + at);
                s.x += q.x, s.y += q.y, s.z += q.z, s.w += q.w;
            }
            if constexpr (sizeof(OT) == 4) {
                *reinterpret_cast<float4 *>(out + at) = s;
            } else {
                const bf16x2 lo = {(__bf16)s.x, (__bf16)s.y}, hi = {(__bf16)s.z, (__bf16)s.w};
                *reinterpret_cast<uint2 *>(out + at) =
                    make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
            }
        }
        return;
    }
    for (; at < count; at += stride) {
        for (int64_t i = at; i < at + 4 && i < count; ++i) {
            float s = part[i];
            for (int n = 1; n < splits; ++n) s += part[n * count + i];
            put(out, i, s);
        }
    }
}

// How A enters: as stored (bf16 grad_y), or the pieces of fp32 values in each tile size.
enum CodesKind { kStored, kWeight32, kWeight16, kInput32 };  // kWeight16: grad_w in bf16
template <int KIND>
struct KindOf {
    static constexpr bool kHalf = KIND != kStored;  // fp16 in large tiles, kLarge pieces
    static constexpr int kLarge = KIND == kStored || KIND == kWeight16 ? 1 : 2;
    static constexpr int kExact = KIND == kStored ? 1 : KIND == kWeight16 ? 2 : 3;  // bf16 pieces
};

// How a product runs: 256 x 256 tiles or 64 x 64 ones, and the workgroups that share
// a tile's slices where there are few tiles: whichever takes the least time by a model
// whose constants were fitted to timed problems of 8 to 4096 tokens. Over 21716 others of
// 8 to 4096 tokens and up to 4096 x 21000 weights, each timed with both tiles and every number
// of workgroups below, what it picks takes 1.5 to 1.8% (weight gradients), 2.3% (input
// gradients of fp32) and 3.4% (of bf16) more on average than the fastest choice, 8 to 15%
// for one in twenty, and 1.74 times at worst (an unaligned weight gradient, 71 us for 41).
//   Small tiles: us for 64 contraction indexes with one workgroup on a compute unit, with
//   more, and for each where they fill the card; large ones: us for a round of one for each
//   compute unit. What a workgroup does besides counts as so many slices more. Rows that
//   are loaded unaligned take a factor.
//   Partial sums: a launch, and 5 TB/s; the search for the largest values of fp16 pieces: a
//   launch, and A read at 3 TB/s.
struct CodesPlan {
    bool large;
    int splits;
};
CodesPlan codes_plan(int64_t I, int64_t J, int64_t P, int kind) {
    static const struct { double one, more, full, start, ragged, large, large_start, large_ragged; } kCost[4] = {
        {0.43, 0.59, 0.33, 4.55, 1.63, 1.73, 3.05, 1.69},
        {1.59, 2.22, 1.09, 0.81, 1.26, 3.60, 2.83, 1.46},
        {0.81, 1.05, 0.70, 1.60, 1.69, 2.22, 1.89, 2.52},
        {0.73, 0.93, 0.60, 3.36, 1.52, 1.94, 2.52, 2.05}};
    const auto &c = kCost[kind];
    const bool weight = kind == kWeight32 || kind == kWeight16;
    const bool ragged = weight ? I % 8 != 0 || J % 16 != 0 : P % 8 != 0;
    const double slices = (double)((P + 63) / 64), out = (double)I * (double)J;
    const double peaks = kind == kStored ? 0.0 : 4.0 + (double)I * (double)P * (kind == kInput32 ? 4e-6 : 2e-6) / 3;
    auto tiles = [&](int64_t side) { return (double)((I + side - 1) / side) * (double)((J + side - 1) / side); };
    // (the search for columns' largest values takes eight of them at a time)
    const bool fits = out >= 32768 && (!weight || I >= 8);
    CodesPlan best{false, 1};
    double least = 1e300;
    for (int n : {1, 2, 3, 4, 6, 8, 12, 16}) {
        if (n > 1 && (n > slices || n * out > 125e6)) break;  // (half a gigabyte of partial sums)
        const double share = std::ceil(slices / n), sums = n > 1 ? 2.5 + out * 1.6e-6 * n : 0.0;
        const double large = std::ceil(tiles(256) * n / 256) * (share + c.large_start) * c.large *
                                 (ragged ? c.large_ragged : 1.0) + peaks + sums;
        const double each = tiles(64) * n / 256;
        const double small = (share + c.start) * std::fmax(each <= 1 ? c.one : c.more, c.full * each) *
                                 (ragged ? c.ragged : 1.0) + sums;
        if (fits && large < least) least = large, best = {true, n};
        if (small < least) least = small, best = {false, n};
    }
    return best;
}
constexpr int64_t kPeakRuns = 64;  // of at least 32 tokens, which a workgroup loads at once
int64_t peak_runs(int64_t M) { return M < 32 * kPeakRuns ? (M + 31) / 32 : kPeakRuns; }
// Floats of partial sums; behind them the largest values and the least, in pairs.
int64_t codes_partials(const CodesPlan &p, int64_t I, int64_t J) {
    return p.splits > 1 ? ((int64_t)p.splits * I * J + 3) / 4 * 4 : 0;
}
size_t codes_workspace(int64_t I, int64_t J, int64_t P, int kind) {
    const CodesPlan p = codes_plan(I, J, P, kind);
    const int64_t peaks = !p.large || kind == kStored ? 0 : 2 * (kind == kInput32 ? I : peak_runs(P) * I);
    return (size_t)(codes_partials(p, I, J) + peaks) * sizeof(float);
}

template <typename T, bool A_T, int BSRC, int NP, bool HALF, int EXACT, typename GT, typename OT>
hipError_t launch_codes(CodesArgs a, bool vec, hipStream_t s) {
    using S = Stage<T, A_T, BSRC, (EXACT > NP ? EXACT : NP)>;
    a.tiles_i = (int)((a.I + T::BI - 1) / T::BI);
    a.tiles_j = (int)((a.J + T::BJ - 1) / T::BJ);
    const int64_t blocks = ((int64_t)a.tiles_i * a.tiles_j * a.splits + kXcds - 1) / kXcds * kXcds;
    auto go = [&](auto kern, LdsFlag *flag) {
        hipError_t e = allow_dynamic_lds(kern, S::SMEM, flag);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(T::kThreads), S::SMEM, s, a);
        return hipGetLastError();
    };
    static LdsFlag lds_raised[2];
    if (vec) return go(codes_gemm_kernel<T, A_T, BSRC, NP, HALF, EXACT, true, GT, OT>, &lds_raised[1]);
    return go(codes_gemm_kernel<T, A_T, BSRC, NP, HALF, EXACT, false, GT, OT>, &lds_raised[0]);
}

// The largest |A(i, .)| and the least that is not zero, in a.peak.
template <bool A_T, typename GT>
hipError_t launch_peaks(const CodesArgs &a, uint2 *peak, hipStream_t s) {
    if constexpr (A_T) {
        const GT *g = static_cast<const GT *>(a.A);
        const dim3 grid((unsigned)((a.I + 255) / 256), (unsigned)a.peaks);
        if (a.I % 8 == 0)
            hipLaunchKernelGGL((codes_peak_cols_kernel<GT, true>), grid, dim3(256), 0, s, g, a.scale, a.P, a.I, peak);
        else
            hipLaunchKernelGGL((codes_peak_cols_kernel<GT, false>), grid, dim3(256), 0, s, g, a.scale, a.P, a.I, peak);
    } else {
        // (2^24 workgroups of 256 would be one thread more than a launch can count)
        const int64_t rows = a.I < 1 << 20 ? a.I : 1 << 20;
        hipLaunchKernelGGL(codes_peak_rows_kernel, dim3((unsigned)rows), dim3(256), 0, s,
                           static_cast<const float *>(a.A), a.I, a.P, peak);
    }
    return hipGetLastError();
}

template <int KIND, int BSRC, typename GT, typename OT>
hipError_t launch_codes_kind(CodesArgs a, bool vec, float *workspace, hipStream_t s) {
    using K = KindOf<KIND>;
    constexpr bool A_T = KIND == kWeight32 || KIND == kWeight16;
    using Large = Tile<256, 256, KIND == kStored ? 64 : 32, 2, 4>;
    // (a stage of three pieces of a [p][i] tile of 64 would leave one workgroup to a
    // compute unit: 1024 tiles 1.1 us each and none side by side)
    using Small = Tile<64, 64, KIND == kWeight32 ? 32 : 64, 2, 2>;
    static_assert(Large::BP <= 64 && Small::BP <= 64, "the plan's slices of 64: a workgroup has at least one");
    const CodesPlan plan = codes_plan(a.I, a.J, a.P, KIND);
    a.splits = plan.splits;
    if constexpr (K::kHalf) {
        if (plan.large) {
            uint2 *peak = reinterpret_cast<uint2 *>(workspace + codes_partials(plan, a.I, a.J));
            a.peaks = A_T ? (int)peak_runs(a.P) : 1;
            a.peak = peak;
            // A value x (of 2^15 at most) is off by 2^-22 x or 2^-25, whichever is more, in two
            // pieces: by max(4, P) 2^-24 of itself at most from this floor on, no more than a sum
            // of P such terms in fp32. In one piece by 2^-11 x or 2^-25: from 2^-14 on 2^-11.
            a.floor = KIND == kWeight16 ? 0x1p-14f : 0.5f / (float)(a.P < 4 ? 4 : a.P);
            const hipError_t e = launch_peaks<A_T, GT>(a, peak, s);
            if (e != hipSuccess) return e;
        }
    }
    OT *out = static_cast<OT *>(a.C);
    auto go = [&](auto *type) {
        using T = Pointee<decltype(type)>;
        return plan.large ? launch_codes<Large, A_T, BSRC, K::kLarge, K::kHalf, K::kExact, GT, T>(a, vec, s)
                          : launch_codes<Small, A_T, BSRC, K::kExact, false, K::kExact, GT, T>(a, vec, s);
    };
    if (plan.splits == 1) return go(out);
    a.C = workspace;
    const hipError_t e = go(workspace);
    if (e != hipSuccess) return e;
    const int64_t count = a.I * a.J, want = (count + 1023) / 1024;
    hipLaunchKernelGGL(codes_sum_kernel<OT>, dim3((unsigned)(want < 8192 ? want : 8192)), dim3(256), 0, s,
                       workspace, out, count, plan.splits);
    return hipGetLastError();
}

}  // namespace

size_t backward_weight_codes_workspace(int64_t M, int64_t N, int64_t K, int gw_dtype) {
    return codes_workspace(N, K, M, gw_dtype == kF32 ? kWeight32 : kWeight16);
}
size_t backward_input_segmented_workspace(int64_t M, int64_t N, int64_t K, int gy_dtype) {
    return codes_workspace(M, K, N, gy_dtype == kF32 ? kInput32 : kStored);
}

hipError_t launch_backward_weight_codes(const void *grad_y, int gy_dtype, const int8_t *xq,
                                        const float *scale, int64_t M, int64_t N, int64_t K,
                                        void *grad_w, int gw_dtype, float *workspace,
                                        hipStream_t stream) {
    const CodesArgs a{grad_y, N, xq, K, scale, {}, N, K, M, 0, 0, 1, nullptr, 0, grad_w, 0.f};
    const bool vec = N % 8 == 0 && K % 16 == 0;
    return typed(gy_dtype, [&](auto g) {
        using GT = Pointee<decltype(g)>;
        if (gw_dtype == kF32)
            return launch_codes_kind<kWeight32, kBCodes8, GT, float>(a, vec, workspace, stream);
        return launch_codes_kind<kWeight16, kBCodes8, GT, uint16_t>(a, vec, workspace, stream);
    });
}

hipError_t launch_backward_input_segmented(const void *grad_y, int gy_dtype, const uint8_t *packed,
                                           int layout, const GammaMap &gamma, int64_t M, int64_t N,
                                           int64_t K, void *grad_x, int gx_dtype, float *workspace,
                                           hipStream_t stream) {
    const CodesArgs a{grad_y, N, packed, row_bytes_of(layout, K), nullptr, gamma, M, K, N,
                      0, 0, 1, nullptr, 0, grad_x, 0.f};
    bool vec = N % 8 == 0;
    for (int s = 0; s + 1 < gamma.nseg; ++s) vec = vec && gamma.bound[s] % 8 == 0;
    auto go = [&](auto src_c) {
        constexpr int B = decltype(src_c)::value;
        return typed(gx_dtype, [&](auto o) {
            using OT = Pointee<decltype(o)>;
            if (gy_dtype == kF32)
                return launch_codes_kind<kInput32, B, float, OT>(a, vec, workspace, stream);
            return launch_codes_kind<kStored, B, uint16_t, OT>(a, vec, workspace, stream);
        });
    };
    switch (layout) {
        case kLayout2Bit: return go(std::integral_constant<int, kBPacked2>{});
        case kLayoutBase3: return go(std::integral_constant<int, kBPacked3>{});
        default: return go(std::integral_constant<int, kBPacked1>{});
    }
}

}  // namespace bl
