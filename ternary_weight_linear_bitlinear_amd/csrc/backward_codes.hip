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

// Block tile BI x BJ outputs, contraction slice BP per stage, 8 waves as 2 x 4.
template <bool A_T, int BSRC, int NP, int BI_>
struct CodesCfg {
    static constexpr int BI = BI_, BJ = 256, BP = NP == 1 ? 64 : 32;
    static constexpr int WI = 2, WJ = 4;
    static constexpr int kThreads = 64 * WI * WJ;
    static constexpr int FI = BI / WI / 32, FJ = BJ / WJ / 32;
    static constexpr int KSTEPS = BP / 16;
    // Padded rows: of a [i][p] tile by 16 bytes, which puts 16 rows of 16-byte reads on
    // distinct banks; of [p][*] tiles by 64, which keeps the four rows of a
    // transposing load apart.
    static constexpr int LD_A = A_T ? BI * 2 + 64 : BP * 2 + 16;
    static constexpr int LD_B = BJ * 2 + 64;
    static constexpr int PLANE = A_T ? BP * LD_A : BI * LD_A;  // one piece of A
    static constexpr int STAGE = NP * PLANE + BP * LD_B;
    static constexpr int LUT = BSRC == kBPacked3 ? 256 * 8 : 0;
    static constexpr int SMEM = 2 * STAGE + LUT;
    static_assert(SMEM <= (int)kLdsBytesPerCu, "two stages in LDS");
};

// Eight consecutive elements as fp32 bits, from any address; elements from `end` on
// (counted from p) are zero and not read.
template <typename T>
__device__ __forceinline__ void load8_any(const T *p, int64_t end, Raw8<T> &r) {
    if (end >= 8) {
        load_any(p, r);
        return;
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < end ? Elem<T>::get(p, e) : 0.f;
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

// VEC: A's rows and segments begin at multiples of 8 elements, xq's at multiples of 16.
template <bool A_T, int BSRC, int NP, int BI_, bool VEC, typename GT, typename OT>
__global__ __launch_bounds__((CodesCfg<A_T, BSRC, NP, BI_>::kThreads)) void codes_gemm_kernel(
    const CodesArgs a) {
    using G = CodesCfg<A_T, BSRC, NP, BI_>;
    static_assert(A_T == (BSRC == kBCodes8), "grad_w from INT8 codes, grad_x from packed ones");
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint64_t *lut = reinterpret_cast<uint64_t *>(smem + 2 * G::STAGE);  // base-3 only

    const int ntiles = a.tiles_i * a.tiles_j;
    const int per_xcd = (ntiles + kXcds - 1) / kXcds;
    const int t = (blockIdx.x % kXcds) * per_xcd + blockIdx.x / kXcds;
    if (t >= ntiles) return;
    const int64_t i0 = (int64_t)(t / a.tiles_j) * G::BI;
    const int64_t j0 = (int64_t)(t % a.tiles_j) * G::BJ;
    const int tid = threadIdx.x;
    const int wave = tid / 64, lane = tid % 64;
    const int wi = wave / G::WJ, wj = wave % G::WJ;

    // Segments in the order of |gamma|: where they begin and end, and the factor
    // that the sums take before the segment's own terms.
    __shared__ int64_t seg_begin[kMaxSegments], seg_end[kMaxSegments];
    __shared__ float seg_ratio[kMaxSegments + 1];
    const int nseg = A_T ? 1 : a.gm.nseg;
    if constexpr (!A_T) {
        if (tid < nseg) {
            const float mine = a.gm.g[tid];
            int rank = 0;
            float before = 0.f;  // the largest |gamma| that goes before
            float signed_before = 0.f;
            for (int s = 0; s < nseg; ++s) {
                const float g = a.gm.g[s];
                if (fabsf(g) < fabsf(mine) || (fabsf(g) == fabsf(mine) && s < tid)) {
                    ++rank;
                    if (fabsf(g) >= before) before = fabsf(g), signed_before = g;
                }
            }
            seg_begin[rank] = tid == 0 ? 0 : a.gm.bound[tid - 1];
            seg_end[rank] = tid == nseg - 1 ? a.P : a.gm.bound[tid];
            seg_ratio[rank] = mine == 0.f ? 1.0f : signed_before / mine;
            if (rank == nseg - 1) seg_ratio[nseg] = mine;
        }
        if constexpr (BSRC == kBPacked3) {
            if (tid < 256) lut[tid] = base3_field_entry((uint32_t)tid);
        }
        __syncthreads();
    }

    // ---- global -> registers, one contraction slice per stage -------------------
    constexpr int A_ROW = A_T ? G::BI / 8 : G::BP / 8;  // chunks of eight in a tile row
    constexpr int A_CH = G::BI * G::BP / 8 / G::kThreads;
    static_assert(A_CH * 8 * G::kThreads == G::BI * G::BP, "whole chunks for every thread");
    Raw8<GT> a_reg[A_CH];
    float a_scale[A_T ? A_CH : 1];
    bool a_ok[A_CH];
    v4i b_reg;  // grad_w: 16 codes of one token; packed: as load_packed leaves them
    bool b_ok = false;
    const GT *A = static_cast<const GT *>(a.A);

    // A piece outside the matrix reads a valid address and is zeroed when it is stored to
    // LDS. (B needs no zeros: its rows past the slice meet zeros of A, its columns past
    // J outputs that are not stored.)
    auto load_stage = [&](int64_t p0, int64_t p1) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < A_CH; ++c) {
            const int q = tid + c * G::kThreads;
            const int64_t p = p0 + (A_T ? q / A_ROW : 8 * (q % A_ROW));
            const int64_t i = i0 + (A_T ? 8 * (q % A_ROW) : q / A_ROW);
            a_ok[c] = p < p1 && i < a.I;
            const GT *src = A + (a_ok[c] ? (A_T ? p * a.lda + i : i * a.lda + p) : 0);
            if constexpr (VEC) {
                a_reg[c].load(src);
            } else {
                // (nothing of a piece outside is used: none of it is read)
                load8_any(src, !a_ok[c] ? 0 : A_T ? a.I - i : p1 - p, a_reg[c]);
            }
            if constexpr (A_T) a_scale[c] = a.scale[p < p1 ? p : p1 - 1];
        }
        const uint8_t *B = static_cast<const uint8_t *>(a.B);
        if constexpr (BSRC == kBCodes8) {
            static_assert(G::BP * G::BJ == 16 * G::kThreads, "16 codes for every thread");
            const int64_t p = p0 + tid / 16, j = j0 + 16 * (tid % 16);
            const bool ok = p < p1 && j < a.J;
            const int8_t *src = reinterpret_cast<const int8_t *>(B) + (ok ? p * a.ldb + j : 0);
            if constexpr (VEC) {
                b_reg = *reinterpret_cast<const v4i *>(src);
            } else if (ok && j + 16 <= a.J) {
                b_reg = load16_any(src);
            } else {
                uint32_t d[4] = {0u, 0u, 0u, 0u};
                if (ok) {
                    for (int e = 0; e < 16; ++e)
                        if (j + e < a.J) d[e / 4] |= (uint32_t)(uint8_t)src[e] << (8 * (e % 4));
                }
                b_reg = v4i{(int)d[0], (int)d[1], (int)d[2], (int)d[3]};
            }
        } else {
            // 32 codes of one weight row for each of 8 BP threads
            if (tid >= 8 * G::BP) return;
            const int64_t p = p0 + tid / 8, c0 = j0 + 32 * (tid % 8);
            const bool row_ok = p < p1;
            const uint8_t *row = B + (row_ok ? p : p0) * a.ldb;
            if constexpr (BSRC == kBPacked2) {
                b_ok = c0 / 4 + 8 <= a.ldb;
                const uint2 v = *reinterpret_cast<const uint2 *>(row + (b_ok ? c0 / 4 : 0));
                b_reg = v4i{(int)v.x, (int)v.y, 0, 0};
            } else if constexpr (BSRC == kBPacked1) {
                b_ok = c0 / 8 + 4 <= a.ldb;
                b_reg = v4i{(int)*reinterpret_cast<const uint32_t *>(row + (b_ok ? c0 / 8 : 0)), 0, 0, 0};
            } else {
                // the eight bytes of codes c0 .. c0 + 31 lie in three dwords (rows are
                // whole dwords; those past the row are five zero codes a byte)
                const int64_t b0 = c0 / 5, al = b0 & ~(int64_t)3;
                uint32_t d[3];
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    d[i] = al + 4 * i < a.ldb ? *reinterpret_cast<const uint32_t *>(row + al + 4 * i)
                                              : 0x79797979u;
                const uint32_t sh = (uint32_t)(b0 - al);
                b_reg = v4i{(int)__builtin_amdgcn_alignbyte(d[1], d[0], sh),
                            (int)__builtin_amdgcn_alignbyte(d[2], d[1], sh), (int)(c0 - 5 * b0), 0};
            }
        }
    };

    // ---- registers -> LDS -------------------------------------------------------
    auto store_a = [&](uint8_t *st) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < A_CH; ++c) {
            const int q = tid + c * G::kThreads;
            uint8_t *dst = st + (q / A_ROW) * G::LD_A + 16 * (q % A_ROW);
            const v4i z = {0, 0, 0, 0};
            if constexpr (NP == 1) {
                *reinterpret_cast<v4i *>(dst) = a_ok[c] ? __builtin_bit_cast(v4i, a_reg[c].a) : z;
            } else {
                float v[8];
                a_reg[c].widen(v);
                if constexpr (A_T) {
                    const float f = a_scale[c] / 127.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= f;
                }
                // (a piece of the remainder of the piece before)
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    v4i w;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = (int)top_halves(__float_as_uint(v[2 * e]), __float_as_uint(v[2 * e + 1]));
                    *reinterpret_cast<v4i *>(dst + n * G::PLANE) = a_ok[c] ? w : z;
                    if (n + 1 < NP) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[e] -= __uint_as_float(__float_as_uint(v[e]) & 0xFFFF0000u);
                    }
                }
            }
        }
    };
    auto store_b = [&](uint8_t *st) __attribute__((always_inline)) {
        uint8_t *Bs = st + NP * G::PLANE;
        if constexpr (BSRC == kBCodes8) {
            uint8_t *dst = Bs + (tid / 16) * G::LD_B + 32 * (tid % 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4i w;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = 8 * h + 2 * e;
                    const float lo = (float)(int8_t)((uint32_t)b_reg[at / 4] >> (8 * (at % 4)));
                    const float hi = (float)(int8_t)((uint32_t)b_reg[at / 4] >> (8 * (at % 4 + 1)));
                    w[e] = (int)top_halves(__float_as_uint(lo), __float_as_uint(hi));
                }
                *reinterpret_cast<v4i *>(dst + 16 * h) = w;
            }
            return;
        }
        if (tid >= 8 * G::BP) return;
        uint8_t *dst = Bs + (tid / 8) * G::LD_B + 64 * (tid % 8);
        uint32_t d[16];
        if constexpr (BSRC == kBPacked1) {
            // bit t of byte i is code 4 t + i; u = 2 bit picks -1 or +1
#pragma unroll
            for (int t = 0; t < 8; ++t)
                field_to_bf16((((uint32_t)b_reg[0] >> t) & 0x01010101u) << 1, d[2 * t], d[2 * t + 1]);
        } else if constexpr (BSRC == kBPacked3) {
            uint32_t f[8];
            base3_fields((uint32_t)b_reg[0], (uint32_t)b_reg[1], b_reg[2], lut, f);
#pragma unroll
            for (int w = 0; w < 8; ++w) field_to_bf16(f[w], d[2 * w], d[2 * w + 1]);
        } else {
            // field s of a word holds its codes 4 s .. 4 s + 3
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    field_to_bf16(((uint32_t)b_reg[w] >> (2 * s)) & 0x03030303u, d[8 * w + 2 * s],
                                  d[8 * w + 2 * s + 1]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4 *>(dst + 16 * q) =
                make_uint4(d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]);
    };

    // ---- fragments ----------------------------------------------------------------
    const int g16 = lane / 16, t16 = lane % 16;
    auto tr_frag = [&](const uint8_t *tile, int ld, int r0, int c0) __attribute__((always_inline)) -> bf16x8 {
        const int row = r0 + 8 * (g16 / 2) + t16 / 4;
        const int col = c0 + 16 * (g16 % 2) + 4 * (t16 % 4);
        const uint8_t *p = tile + row * ld + col * 2;
        const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p));
        const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p + 4 * ld));
        const v8s both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf16x8, both);
    };
    v16f acc[G::FI][G::FJ];
#pragma unroll
    for (int i = 0; i < G::FI; ++i)
#pragma unroll
        for (int j = 0; j < G::FJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    auto compute = [&](const uint8_t *st) __attribute__((always_inline)) {
        const uint8_t *Bs = st + NP * G::PLANE;
#pragma unroll
        for (int ks = 0; ks < G::KSTEPS; ++ks) {
            bf16x8 bb[G::FJ];
#pragma unroll
            for (int j = 0; j < G::FJ; ++j)
                bb[j] = tr_frag(Bs, G::LD_B, 16 * ks, wj * (G::BJ / G::WJ) + j * 32);
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                const uint8_t *As = st + n * G::PLANE;
                bf16x8 af[G::FI];
#pragma unroll
                for (int i = 0; i < G::FI; ++i) {
                    const int ibase = wi * (G::BI / G::WI) + i * 32;
                    if constexpr (A_T)
                        af[i] = tr_frag(As, G::LD_A, 16 * ks, ibase);
                    else
                        af[i] = *reinterpret_cast<const bf16x8 *>(
                            As + (ibase + lane % 32) * G::LD_A + (16 * ks + 8 * (lane / 32)) * 2);
                }
#pragma unroll
                for (int i = 0; i < G::FI; ++i)
#pragma unroll
                    for (int j = 0; j < G::FJ; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[i], bb[j], acc[i][j], 0, 0, 0);
            }
        }
    };

    // ---- the slices of every segment in turn --------------------------------------
    int seg = 0;
    auto begin_of = [&](int s) { return A_T ? (int64_t)0 : seg_begin[s]; };
    auto end_of = [&](int s) { return A_T ? a.P : seg_end[s]; };
    int64_t p = begin_of(0), end = end_of(0);
    load_stage(p, end);
    store_a(smem);
    store_b(smem);
    __syncthreads();
    for (int buf = 0;; buf ^= 1) {
        // the next slice; `fresh`: the first one of its segment
        bool more = true, fresh = false;
        p += G::BP;
        if (p >= end) {
            if (++seg < nseg) {
                p = begin_of(seg);
                end = end_of(seg);
                fresh = true;
            } else {
                more = false;
            }
        }
        if (more) load_stage(p, end);
        compute(smem + buf * G::STAGE);
        if (!more) break;
        if (fresh) {
            const float f = seg_ratio[seg];
#pragma unroll
            for (int i = 0; i < G::FI; ++i)
#pragma unroll
                for (int j = 0; j < G::FJ; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[i][j][r] *= f;
        }
        store_a(smem + (buf ^ 1) * G::STAGE);
        store_b(smem + (buf ^ 1) * G::STAGE);
        lds_barrier();
    }

    // ---- epilogue: lane holds D[i][j] for j = lane % 32 and
    // i = 8 (r / 4) + 4 (lane / 32) + r % 4, register r
    const float alpha = A_T ? 1.0f : seg_ratio[nseg];
    OT *C = static_cast<OT *>(a.C);
#pragma unroll
    for (int fi = 0; fi < G::FI; ++fi)
#pragma unroll
        for (int fj = 0; fj < G::FJ; ++fj) {
            const int64_t j = j0 + wj * (G::BJ / G::WJ) + fj * 32 + lane % 32;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int64_t i =
                    i0 + wi * (G::BI / G::WI) + fi * 32 + 8 * (r / 4) + 4 * (lane / 32) + r % 4;
                if (i < a.I && j < a.J) put(C, i * a.J + j, A_T ? acc[fi][fj][r] : acc[fi][fj][r] * alpha);
            }
        }
}

template <bool A_T, int BSRC, int NP, int BI, bool VEC, typename GT, typename OT>
hipError_t launch_codes(CodesArgs a, hipStream_t s) {
    using G = CodesCfg<A_T, BSRC, NP, BI>;
    a.tiles_i = (int)((a.I + G::BI - 1) / G::BI);
    a.tiles_j = (int)((a.J + G::BJ - 1) / G::BJ);
    const int64_t blocks = ((int64_t)a.tiles_i * a.tiles_j + kXcds - 1) / kXcds * kXcds;
    auto kern = codes_gemm_kernel<A_T, BSRC, NP, BI, VEC, GT, OT>;
    static LdsFlag lds_raised{0};
    hipError_t e = allow_dynamic_lds(kern, G::SMEM, &lds_raised);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(G::kThreads), G::SMEM, s, a);
    return hipGetLastError();
}

template <bool A_T, int BSRC, int NP, typename GT, typename OT>
hipError_t launch_codes_sized(const CodesArgs &a, bool vec, hipStream_t s) {
    // half-height tiles where 256 x 256 ones would leave compute units without one
    const int64_t whole = ((a.I + 255) / 256) * ((a.J + 255) / 256);
    if (whole < 256)
        return vec ? launch_codes<A_T, BSRC, NP, 128, true, GT, OT>(a, s)
                   : launch_codes<A_T, BSRC, NP, 128, false, GT, OT>(a, s);
    return vec ? launch_codes<A_T, BSRC, NP, 256, true, GT, OT>(a, s)
               : launch_codes<A_T, BSRC, NP, 256, false, GT, OT>(a, s);
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
