// Backward of the products' extended epilogue:
//   grad_z = grad_y * act'(z),  grad_bias = sum_m grad_z,  grad_residual = res_scale * grad_y.
// act' is recomputed from the stored pre-activation z; grad_bias sums the
// unrounded grad_z. Memory-bound: grad_y and z are read once, grad_z (and
// grad_residual) written once.
//
// A workgroup takes 8 PIECES columns of a run of rows: PIECES threads side by
// side hold eight columns each, 256 / PIECES rows at a time, and keep their
// columns' sums in registers; the rows of threads are added through LDS. Wide
// workgroups (32 pieces, 512 bytes of a bf16 row) with runs enough to fill the
// card write one partial sum per run and column, which a second kernel adds in
// fp64. Up to kOneRunRows tokens narrow ones (8 pieces, 32 rows at a time) take
// all rows and write grad_bias themselves: one launch.
#include "activation.hpp"
#include "bl_internal.hpp"
#include "device_util.hpp"
#include "row_share.hpp"

namespace bl {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kRunRows = 512;  // at most, so that the fp32 sums stay short
constexpr int64_t kOneRunRows = 128;
constexpr int kWide = 32, kNarrow = 8;

template <typename GT, typename ZT, typename OT, int PIECES, bool VEC>
__global__ __launch_bounds__(kThreads) void epilogue_grad_kernel(const EpilogueGradArgs a,
                                                                 int64_t runs) {
    constexpr int kRows = kThreads / PIECES, kCols = 8 * PIECES, kUnroll = 4;
    __shared__ float red[kRows][kCols];
    const int r = threadIdx.x / PIECES;
    const int64_t n0 = (int64_t)blockIdx.x * kCols;
    const int left = (int)(a.N - n0 < kCols ? a.N - n0 : kCols);
    const Share<1, VEC> sh{left, (int)threadIdx.x % PIECES, PIECES};
    const int64_t m0 = a.M * blockIdx.y / runs, m1 = a.M * (blockIdx.y + 1) / runs;
    const bool slope = a.act != kActNone;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int64_t m = m0 + r; m < m1; m += kUnroll * kRows) {
        RowRegs<GT, 1, VEC> rg[kUnroll];
        RowRegs<ZT, 1, VEC> rz[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {  // rows past the run read its last one
            const int64_t mu = m + u * kRows < m1 ? m + u * kRows : m1 - 1;
            rg[u].load(static_cast<const GT *>(a.grad_y) + mu * a.N + n0, sh);
            if (slope) rz[u].load(static_cast<const ZT *>(a.z) + mu * a.N + n0, sh);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t mu = m + u * kRows;
            if (mu >= m1) break;
            const int64_t at = mu * a.N + n0;
            float g[8];
            rg[u].widen(0, sh, g);
            if (a.grad_residual) {
                float t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = a.res_scale * g[e];
                store_share(static_cast<GT *>(a.grad_residual) + at, 0, sh, t);
            }
            if (slope) {
                float z[8];
                rz[u].widen(0, sh, z);
                times_slope(g, z, a.act);
            }
            if (a.grad_z) store_share(static_cast<OT *>(a.grad_z) + at, 0, sh, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += g[e];
        }
    }
    if (!a.grad_bias) return;
    const int start = sh.start(0), skip = sh.skip(0);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e >= skip) red[r][start + e] = s[e];
    __syncthreads();
    if ((int)threadIdx.x >= left) return;
    float t = red[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kRows; ++i) t += red[i][threadIdx.x];
    float *out = runs == 1 ? a.grad_bias : a.workspace + blockIdx.y * a.N;
    out[n0 + threadIdx.x] = t;
}

// Fewer than eight columns: a thread for each, over a run of rows.
template <typename GT, typename ZT, typename OT>
__global__ __launch_bounds__(64) void epilogue_grad_few_kernel(const EpilogueGradArgs a,
                                                               int64_t runs) {
    const int64_t n = threadIdx.x;
    if (n >= a.N) return;
    const int64_t m0 = a.M * blockIdx.x / runs, m1 = a.M * (blockIdx.x + 1) / runs;
    float s = 0.f;
    for (int64_t m = m0; m < m1; ++m) {
        const int64_t at = m * a.N + n;
        const float y = Elem<GT>::get(static_cast<const GT *>(a.grad_y), at);
        if (a.grad_residual) put(static_cast<GT *>(a.grad_residual), at, a.res_scale * y);
        float g[1] = {y};
        if (a.act != kActNone) {
            const float z[1] = {Elem<ZT>::get(static_cast<const ZT *>(a.z), at)};
            times_slope(g, z, a.act);
        }
        if (a.grad_z) put(static_cast<OT *>(a.grad_z), at, g[0]);
        s += g[0];
    }
    if (a.grad_bias) (runs == 1 ? a.grad_bias : a.workspace + blockIdx.x * a.N)[n] = s;
}

// grad_bias from the runs' partials, in fp64: 32 columns per workgroup, the runs
// over its eight rows of threads.
__global__ __launch_bounds__(kThreads) void epilogue_grad_sums_kernel(const float *part,
                                                                      float *out, int64_t N,
                                                                      int64_t runs) {
    __shared__ double red[8][33];
    const int c = threadIdx.x % 32, r = threadIdx.x / 32;
    const int64_t n = (int64_t)blockIdx.x * 32 + c;
    double s = 0.0;
    if (n < N) {
#pragma unroll 8
        for (int64_t p = r; p < runs; p += 8) s += (double)part[p * N + n];
    }
    red[r][c] = s;
    __syncthreads();
    if (r > 0 || n >= N) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][c];
    out[n] = (float)s;
}

}  // namespace

hipError_t launch_run_sums(const float *part, float *out, int64_t N, int64_t runs, hipStream_t stream) {
    hipLaunchKernelGGL(epilogue_grad_sums_kernel, dim3((unsigned)((N + 31) / 32)), dim3(kThreads), 0,
                       stream, part, out, N, runs);
    return hipGetLastError();
}

int64_t epilogue_grad_parts(int64_t M, int64_t N) {
    if (M <= kOneRunRows) return 1;
    const int64_t wide = (N + 8 * kWide - 1) / (8 * kWide);
    int64_t runs = (2048 + wide - 1) / wide;  // eight workgroups for each of 256 compute units
    if (runs > (M + 31) / 32) runs = (M + 31) / 32;  // one unrolled step of rows each, at least
    if (runs < (M + kRunRows - 1) / kRunRows) runs = (M + kRunRows - 1) / kRunRows;
    return runs;
}

hipError_t launch_epilogue_backward(const EpilogueGradArgs &a, hipStream_t stream) {
    const int64_t runs = epilogue_grad_parts(a.M, a.N);
    return typed(a.gy_dtype, [&](auto g) {
        return typed(a.z_dtype, [&](auto z) {
            return typed(a.gz_dtype, [&](auto o) {
                using GT = Pointee<decltype(g)>;
                using ZT = Pointee<decltype(z)>;
                using OT = Pointee<decltype(o)>;
                auto go = [&](auto pieces_c, auto vec_c) {
                    constexpr int P = decltype(pieces_c)::value;
                    const dim3 grid((unsigned)((a.N + 8 * P - 1) / (8 * P)), (unsigned)runs);
                    hipLaunchKernelGGL((epilogue_grad_kernel<GT, ZT, OT, P, decltype(vec_c)::value>),
                                       grid, dim3(kThreads), 0, stream, a, runs);
                    return hipGetLastError();
                };
                auto pieces = [&](auto vec_c) {
                    return runs == 1 ? go(std::integral_constant<int, kNarrow>{}, vec_c)
                                     : go(std::integral_constant<int, kWide>{}, vec_c);
                };
                hipError_t e;
                if (a.N < 8) {
                    hipLaunchKernelGGL((epilogue_grad_few_kernel<GT, ZT, OT>), dim3((unsigned)runs),
                                       dim3(64), 0, stream, a, runs);
                    e = hipGetLastError();
                } else {
                    e = a.N % 8 == 0 ? pieces(std::true_type{}) : pieces(std::false_type{});
                }
                if (e != hipSuccess || !a.grad_bias || runs == 1) return e;
                return launch_run_sums(a.workspace, a.grad_bias, a.N, runs, stream);
            });
        });
    });
}

}  // namespace bl
