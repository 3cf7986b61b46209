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
// An fp32 value of A is taken as three bf16 pieces (exact, f32_piece_bits), which are
// multiplied by the same fragment of B one after the other: v is one fp32 rounding of
// its product, each term of grad_w exact beyond it. grad_w in bf16 takes two pieces
// (v to within 2^-15), far below its own rounding of 2^-8.
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
#include "backward_util.hpp"
#include "bl_internal.hpp"
#include "device_util.hpp"
#include "row_share.hpp"

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
    void *C;  // [I, J]
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
// tiles by 64, which keeps the four rows of a transposing load apart.
template <typename T, bool A_T, int BSRC, int NP>
struct Stage {
    static constexpr int LD_A = A_T ? T::BI * 2 + 64 : T::BP * 2 + 16;
    static constexpr int LD_B = T::BJ * 2 + 64;
    static constexpr int PLANE = A_T ? T::BP * LD_A : T::BI * LD_A;  // one piece of A
    static constexpr int BYTES = NP * PLANE + T::BP * LD_B;
    static constexpr int LUT = BSRC == kBPacked3 ? 256 * 8 : 0;
    static constexpr int SMEM = 2 * BYTES + LUT;
    static_assert(SMEM <= (int)kLdsBytesPerCu, "two stages in LDS");
};

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
template <typename T, bool A_T, int BSRC, int NP, bool VEC, typename GT, typename OT>
__global__ __launch_bounds__(T::kThreads) void codes_gemm_kernel(const CodesArgs a) {
    using S = Stage<T, A_T, BSRC, NP>;
    constexpr int kT = T::kThreads;
    static_assert(A_T == (BSRC == kBCodes8), "grad_w from INT8 codes, grad_x from packed ones");
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint64_t *lut = reinterpret_cast<uint64_t *>(smem + 2 * S::BYTES);  // base-3 only

    const int ntiles = a.tiles_i * a.tiles_j;
    const int per_xcd = (ntiles + kXcds - 1) / kXcds;
    const int t = (blockIdx.x % kXcds) * per_xcd + blockIdx.x / kXcds;
    if (t >= ntiles) return;
    const int64_t i0 = (int64_t)(t / a.tiles_j) * T::BI;
    const int64_t j0 = (int64_t)(t % a.tiles_j) * T::BJ;
    const int tid = threadIdx.x;
    const int wave = tid / 64, lane = tid % 64;
    const int wi = wave / T::WJ, wj = wave % T::WJ;

    // Segments in the order of |gamma|: where they begin and end, and the factor
    // that the sums take before the segment's own terms.
    __shared__ int64_t seg_begin[kMaxSegments], seg_end[kMaxSegments];
    __shared__ float seg_ratio[kMaxSegments + 1];
    const int nseg = A_T ? 1 : a.gm.nseg;
    if constexpr (!A_T) {
        if (tid < nseg) {
            const float mine = a.gm.g[tid];
            int rank = 0;
            float before = 0.f;  // of the largest |gamma| that goes before
            for (int s = 0; s < nseg; ++s) {
                const float g = a.gm.g[s];
                if (fabsf(g) < fabsf(mine) || (fabsf(g) == fabsf(mine) && s < tid)) {
                    ++rank;
                    if (fabsf(g) >= fabsf(before)) before = g;
                }
            }
            seg_begin[rank] = tid == 0 ? 0 : a.gm.bound[tid - 1];
            seg_end[rank] = tid == nseg - 1 ? a.P : a.gm.bound[tid];
            seg_ratio[rank] = mine == 0.f ? 1.0f : before / mine;
            if (rank == nseg - 1) seg_ratio[nseg] = mine;
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
    constexpr int B_EACH = BSRC == kBCodes8 ? 16 : 32, B_ROW = T::BJ / B_EACH;  // codes; threads of a row
    constexpr int B_CH = (T::BP * B_ROW + kT - 1) / kT;
    static_assert(T::BP * B_ROW % kT == 0 || T::BP * B_ROW < kT, "whole rows of B");
    constexpr int B_STEP = kT / B_ROW;
    Raw8<GT> a_reg[A_CH];
    float a_scale[A_T ? A_CH : 1];
    v4i b_reg[B_CH];  // grad_w: 16 codes of one token; packed: as unpacked below
    const int ar = tid / A_ROW, ac = tid % A_ROW;
    const int br = tid / B_ROW, bc = tid % B_ROW;
    const bool b_mine = B_CH > 1 || T::BP * B_ROW >= kT || br < T::BP;
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
    // (packed rows are whole 16-byte pieces, so 2-bit and 1-bit pieces lie wholly in or
    // past them; of base-3 the dwords past a row are taken from its start)
    const int64_t b_first = BSRC == kBPacked3 ? c0 / 5 & ~(int64_t)3 : c0 / kPer;
    constexpr int kWords = BSRC == kBPacked2 ? 2 : BSRC == kBPacked1 ? 1 : 3;
    int b_at[3];  // bytes from the row's start; codes: the first only
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int64_t at = b_first + 4 * i;
        b_at[i] = BSRC == kBCodes8 ? (c0 < a.J ? (int)c0 : 0) : at < a.ldb ? (int)at : 0;
    }
    const int b_shift = BSRC == kBPacked3 ? (int)(c0 / 5 - b_first) : 0;
    const int b_code = BSRC == kBPacked3 ? (int)(c0 % 5) : 0;

    auto load_b = [&](int c, const uint8_t *row) __attribute__((always_inline)) {
        if constexpr (BSRC == kBCodes8) {
            b_reg[c] = VEC ? *reinterpret_cast<const v4i *>(row + b_at[0])
                           : load16_any(reinterpret_cast<const int8_t *>(row) + b_at[0]);
        } else if constexpr (BSRC == kBPacked2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(row + b_at[0]);
            b_reg[c] = v4i{(int)v.x, (int)v.y, 0, 0};
        } else {
            uint32_t d[3] = {0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < kWords; ++i) d[i] = *reinterpret_cast<const uint32_t *>(row + b_at[i]);
            b_reg[c] = v4i{(int)d[0], (int)d[1], (int)d[2], 0};
        }
    };
    // The slice [p0, p0 + BP) of a segment that ends at p1. A whole slice has no
    // checks; unaligned pieces of [p][*] tiles at the right edge run on into the next
    // rows, which have to be there.
    auto load_stage = [&](int64_t p0, int64_t p1) __attribute__((always_inline)) {
        const int64_t past = VEC || !A_T ? 0 : 16;  // rows that hold 16 elements, at least
        if (p0 + T::BP + past <= p1) {
#pragma unroll
            for (int c = 0; c < A_CH; ++c) {
                const GT *at = A_T ? a_base[0] + (p0 + c * A_STEP) * a.lda : a_base[A_T ? 0 : c] + p0;
                const GT *src = reinterpret_cast<const GT *>(reinterpret_cast<const char *>(at) +
                                                             a_off[A_T ? 0 : c]);
                if constexpr (VEC) a_reg[c].load(src);
                else load_any(src, a_reg[c]);
                if constexpr (A_T) a_scale[c] = a.scale[p0 + ar + c * A_STEP];
            }
            if (b_mine) {
#pragma unroll
                for (int c = 0; c < B_CH; ++c) load_b(c, B + (p0 + br + c * B_STEP) * a.ldb);
            }
            return;
        }
        // the end of a segment: A is zero past it (B need not be)
#pragma unroll
        for (int c = 0; c < A_CH; ++c) {
            const int row = ar + c * A_STEP;
            const int64_t p = p0 + (A_T ? row : 8 * ac), i = i0 + (A_T ? 8 * ac : row);
            const bool ok = p < p1 && i < a.I;
            const int64_t left = !ok ? 0 : A_T ? a.I - i : p1 - p;
            load8_some(A + (ok ? (A_T ? p * a.lda + i : i * a.lda + p) : 0), left, a_reg[c]);
            if constexpr (A_T) a_scale[c] = a.scale[p < p1 ? p : p1 - 1];
        }
        if (!b_mine) return;
#pragma unroll
        for (int c = 0; c < B_CH; ++c) {
            const int64_t p = p0 + br + c * B_STEP;
            const uint8_t *row = B + (p < p1 ? p : p1 - 1) * a.ldb;
            if constexpr (BSRC == kBCodes8) {
                uint32_t d[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (c0 + e < a.J) d[e / 4] |= (uint32_t)row[c0 + e] << (8 * (e % 4));
                b_reg[c] = v4i{(int)d[0], (int)d[1], (int)d[2], (int)d[3]};
            } else {
                load_b(c, row);
            }
        }
    };

    // ---- registers -> LDS -----------------------------------------------------------
    auto store_a = [&](uint8_t *st, int c) __attribute__((always_inline)) {
        uint8_t *dst = st + (ar + c * A_STEP) * S::LD_A + 16 * ac;
        if constexpr (NP == 1) {
            *reinterpret_cast<v4i *>(dst) = __builtin_bit_cast(v4i, a_reg[c].a);
        } else {
            float v[8];
            a_reg[c].widen(v);
            if constexpr (A_T) {
                const float f = over127(a_scale[c]);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= f;
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
        uint8_t *dst = st + NP * S::PLANE + (br + c * B_STEP) * S::LD_B + 2 * B_EACH * bc;
        uint32_t d[B_EACH / 2];
        if constexpr (BSRC == kBCodes8) {
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const uint32_t w = (uint32_t)b_reg[c][e / 4];
                const float lo = (float)(int8_t)(w >> (8 * (e % 4))), hi = (float)(int8_t)(w >> (8 * (e % 4 + 1)));
                d[e / 2] = top_halves(__float_as_uint(lo), __float_as_uint(hi));
            }
        } else if constexpr (BSRC == kBPacked1) {
            // bit t of byte i is code 4 t + i; u = 2 bit picks -1 or +1
#pragma unroll
            for (int t = 0; t < 8; ++t)
                field_to_bf16((((uint32_t)b_reg[c][0] >> t) & 0x01010101u) << 1, d[2 * t], d[2 * t + 1]);
        } else if constexpr (BSRC == kBPacked3) {
            // the eight bytes of codes c0 .. c0 + 31 lie in three dwords
            uint32_t f[8];
            base3_fields(__builtin_amdgcn_alignbyte(b_reg[c][1], b_reg[c][0], b_shift),
                         __builtin_amdgcn_alignbyte(b_reg[c][2], b_reg[c][1], b_shift), b_code, lut, f);
#pragma unroll
            for (int w = 0; w < 8; ++w) field_to_bf16(f[w], d[2 * w], d[2 * w + 1]);
        } else {
            // field s of a word holds its codes 4 s .. 4 s + 3
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    field_to_bf16(((uint32_t)b_reg[c][w] >> (2 * s)) & 0x03030303u, d[8 * w + 2 * s],
                                  d[8 * w + 2 * s + 1]);
        }
#pragma unroll
        for (int q = 0; q < B_EACH / 8; ++q)
            *reinterpret_cast<uint4 *>(dst + 16 * q) =
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
    const int b_lane = NP * S::PLANE + tr_row * S::LD_B + tr_col + wj * (T::BJ / T::WJ) * 2;
    auto a_frag = [&](const uint8_t *st, int ks, int n, int i) __attribute__((always_inline)) -> bf16x8 {
        const uint8_t *p = st + a_lane + n * S::PLANE;
        if constexpr (A_T) return tr_frag(p + 16 * ks * S::LD_A + i * 64, S::LD_A);
        else return *reinterpret_cast<const bf16x8 *>(p + i * 32 * S::LD_A + 32 * ks);
    };
    auto b_frag = [&](const uint8_t *st, int ks, int j) __attribute__((always_inline)) -> bf16x8 {
        return tr_frag(st + b_lane + 16 * ks * S::LD_B + j * 64, S::LD_B);
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
    auto begin_of = [&](int s) { return A_T ? (int64_t)0 : seg_begin[s]; };
    auto end_of = [&](int s) { return A_T ? a.P : seg_end[s]; };
    auto after = [&](Slice s) {  // seg == nseg: none
        s.p += T::BP;
        if (s.p >= s.end && ++s.seg < nseg) s.p = begin_of(s.seg), s.end = end_of(s.seg);
        return s;
    };
    Slice cur{0, begin_of(0), end_of(0)};
    load_stage(cur.p, cur.end);
#pragma unroll
    for (int c = 0; c < A_CH; ++c) store_a(smem, c);
#pragma unroll
    for (int c = 0; c < B_CH; ++c) store_b(smem, c);
    Slice next = after(cur);
    if (next.seg < nseg) load_stage(next.p, next.end);
    __syncthreads();
    constexpr int kGroups = T::KSTEPS * NP;
    for (int buf = 0;; buf ^= 1) {
        const uint8_t *st = smem + buf * S::BYTES;
        uint8_t *to = smem + (buf ^ 1) * S::BYTES;
        const bool more = next.seg < nseg;
        const Slice then = more ? after(next) : next;
        bf16x8 af[2][T::FI], bb[2][T::FJ];
#pragma unroll
        for (int j = 0; j < T::FJ; ++j) bb[0][j] = b_frag(st, 0, j);
#pragma unroll
        for (int i = 0; i < T::FI; ++i) af[0][i] = a_frag(st, 0, 0, i);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int ks = g / NP;
            if (g + 1 < kGroups) {
                const int k1 = (g + 1) / NP, n1 = (g + 1) % NP;
                if (n1 == 0) {
#pragma unroll
                    for (int j = 0; j < T::FJ; ++j) bb[k1 & 1][j] = b_frag(st, k1, j);
                }
#pragma unroll
                for (int i = 0; i < T::FI; ++i) af[(g + 1) & 1][i] = a_frag(st, k1, n1, i);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < T::FI; ++i)
#pragma unroll
                for (int j = 0; j < T::FJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[g & 1][i], bb[ks & 1][j], acc[i][j],
                                                                        0, 0, 0);
            // this group's share of the next stage
            if (more) {
                constexpr int kTasks = A_CH + B_CH;
#pragma unroll
                for (int q = g * kTasks / (kGroups - 1); q < (g + 1) * kTasks / (kGroups - 1); ++q) {
                    if (q < A_CH) store_a(to, q);
                    else if (q < kTasks) store_b(to, q - A_CH);
                }
                if (g == kGroups - 1 && then.seg < nseg) load_stage(then.p, then.end);
            }
        }
        if (!more) break;
        if (next.seg != cur.seg) {
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
        lds_barrier();
    }

    // ---- epilogue: lane holds D[i][j] for j = lane % 32 and
    // i = 8 (r / 4) + 4 (lane / 32) + r % 4, register r
    const float alpha = A_T ? 1.0f : seg_ratio[nseg];
    OT *C = static_cast<OT *>(a.C);
#pragma unroll
    for (int fi = 0; fi < T::FI; ++fi)
#pragma unroll
        for (int fj = 0; fj < T::FJ; ++fj) {
            const int64_t j = j0 + wj * (T::BJ / T::WJ) + fj * 32 + lane % 32;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int64_t i =
                    i0 + wi * (T::BI / T::WI) + fi * 32 + 8 * (r / 4) + 4 * (lane / 32) + r % 4;
                if (i < a.I && j < a.J) put(C, i * a.J + j, A_T ? acc[fi][fj][r] : acc[fi][fj][r] * alpha);
            }
        }
}

template <typename T, bool A_T, int BSRC, int NP, typename GT, typename OT>
hipError_t launch_codes(CodesArgs a, bool vec, hipStream_t s) {
    using S = Stage<T, A_T, BSRC, NP>;
    a.tiles_i = (int)((a.I + T::BI - 1) / T::BI);
    a.tiles_j = (int)((a.J + T::BJ - 1) / T::BJ);
    const int64_t blocks = ((int64_t)a.tiles_i * a.tiles_j + kXcds - 1) / kXcds * kXcds;
    auto go = [&](auto kern, LdsFlag *flag) {
        hipError_t e = allow_dynamic_lds(kern, S::SMEM, flag);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(T::kThreads), S::SMEM, s, a);
        return hipGetLastError();
    };
    static LdsFlag lds_raised[2];
    if (vec) return go(codes_gemm_kernel<T, A_T, BSRC, NP, true, GT, OT>, &lds_raised[1]);
    return go(codes_gemm_kernel<T, A_T, BSRC, NP, false, GT, OT>, &lds_raised[0]);
}

template <bool A_T, int BSRC, int NP, typename GT, typename OT>
hipError_t launch_codes_sized(const CodesArgs &a, bool vec, hipStream_t s) {
    constexpr int BP = NP == 1 ? 64 : 32;
    auto tiles = [&](int64_t bi, int64_t bj) { return ((a.I + bi - 1) / bi) * ((a.J + bj - 1) / bj); };
    if (tiles(256, 256) >= 256) return launch_codes<Tile<256, 256, BP, 2, 4>, A_T, BSRC, NP, GT, OT>(a, vec, s);
    if (tiles(128, 256) >= 128) return launch_codes<Tile<128, 256, BP, 2, 4>, A_T, BSRC, NP, GT, OT>(a, vec, s);
    return launch_codes<Tile<64, 64, 64, 2, 2>, A_T, BSRC, NP, GT, OT>(a, vec, s);
}

}  // namespace

hipError_t launch_backward_weight_codes(const void *grad_y, int gy_dtype, const int8_t *xq,
                                        const float *scale, int64_t M, int64_t N, int64_t K,
                                        void *grad_w, int gw_dtype, hipStream_t stream) {
    CodesArgs a{grad_y, N, xq, K, scale, {}, N, K, M, 0, 0, grad_w};
    const bool vec = N % 8 == 0 && K % 16 == 0;
    return typed(gy_dtype, [&](auto g) {
        using GT = Pointee<decltype(g)>;
        if (gw_dtype == kF32) return launch_codes_sized<true, kBCodes8, 3, GT, float>(a, vec, stream);
        return launch_codes_sized<true, kBCodes8, 2, GT, uint16_t>(a, vec, stream);
    });
}

hipError_t launch_backward_input_segmented(const void *grad_y, int gy_dtype, const uint8_t *packed,
                                           int layout, const GammaMap &gamma, int64_t M, int64_t N,
                                           int64_t K, void *grad_x, int gx_dtype, hipStream_t stream) {
    const CodesArgs a{grad_y, N, packed, row_bytes_of(layout, K), nullptr, gamma, M, K, N, 0, 0, grad_x};
    bool vec = N % 8 == 0;
    for (int s = 0; s + 1 < gamma.nseg; ++s) vec = vec && gamma.bound[s] % 8 == 0;
    auto go = [&](auto src_c) {
        constexpr int B = decltype(src_c)::value;
        return typed(gx_dtype, [&](auto o) {
            using OT = Pointee<decltype(o)>;
            if (gy_dtype == kF32) return launch_codes_sized<false, B, 3, float, OT>(a, vec, stream);
            return launch_codes_sized<false, B, 1, uint16_t, OT>(a, vec, stream);
        });
    };
    switch (layout) {
        case kLayout2Bit: return go(std::integral_constant<int, kBPacked2>{});
        case kLayoutBase3: return go(std::integral_constant<int, kBPacked3>{});
        default: return go(std::integral_constant<int, kBPacked1>{});
    }
}

}  // namespace bl
