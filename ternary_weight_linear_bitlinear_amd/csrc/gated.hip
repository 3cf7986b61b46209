// Backward of the gated products' epilogue, y = act(z_0) * z_1 over the two halves
// of z [M, 2F]:
//   grad_z_0 = grad_y * z_1 * act'(z_0),  grad_z_1 = grad_y * act(z_0),
//   grad_bias = sum_m grad_z.
// z comes as the forward pass stored it, or from its 8-bit checkpoint: codes of
// rows 2m (gate) and 2m + 1 (up) with a scale for each 64 columns. Memory-bound:
// each input is read once, grad_z written once.
//
// The split is that of the plain epilogue's backward pass (epilogue.hip), with the
// two halves of a column in one thread: 8 PIECES columns of a run of rows for each
// workgroup, eight columns of both halves for each thread, column sums in
// registers, the rows of threads added through LDS, and the runs' partial sums by
// a second kernel in fp64. Up to kOneRunRows tokens take one launch.
//
// 2048 x 11008, bf16 in and out, z from its checkpoint: 37.3 us, 93 MB read and 90 MB
// written (what it must), 4.9 TB/s, the rate of a large copy. 100 x 1003 in fp32: 7.0
// us, one unrolled step of rows, their sum through LDS and the launch.
#include "activation.hpp"
#include "bl_internal.hpp"
#include "device_util.hpp"
#include "row_share.hpp"

namespace bl {
namespace {

constexpr int kThreads = 256, kXcds = 8;
constexpr int64_t kRunRows = 512;  // at most, so that the fp32 sums stay short
constexpr int64_t kOneRunRows = 128;
constexpr int kWide = 32, kNarrow = 8;

// A thread's eight columns of one half of z, as stored (ZT float or bf16) or kept
// in 8 bits (ZT int8_t).
template <typename ZT, bool VEC>
struct ZRegs {
    RowRegs<ZT, 1, VEC> r;
    __device__ __forceinline__ void load(const GatedGradArgs &a, int64_t row, int64_t n0,
                                         const Share<1, VEC> &sh, int64_t) {
        r.load(static_cast<const ZT *>(a.z) + row * a.F + n0, sh);
    }
    __device__ __forceinline__ void widen(const Share<1, VEC> &sh, float (&v)[8]) const { r.widen(0, sh, v); }
};
template <bool VEC>
struct ZRegs<int8_t, VEC> {
    Kept8 r;
    __device__ __forceinline__ void load(const GatedGradArgs &a, int64_t row, int64_t n0,
                                         const Share<1, VEC> &sh, int64_t group) {
        load_kept(a.codes + row * a.F + n0, a.code_scale + row * checkpoint_groups(a.F), group, sh, r);
    }
    __device__ __forceinline__ void widen(const Share<1, VEC> &sh, float (&v)[8]) const {
        r.widen(v);
        clear_past(0, sh, v);
    }
};

template <typename GT, typename ZT, typename OT, int PIECES, bool VEC>
__global__ __launch_bounds__(kThreads) void gated_grad_kernel(const GatedGradArgs a, int64_t runs) {
    constexpr int kRows = kThreads / PIECES, kCols = 8 * PIECES, kUnroll = 4;
    __shared__ float red[2][kRows][kCols];
    const int r = threadIdx.x / PIECES;
    // Workgroups are dealt to the XCDs in turn; each XCD takes neighbouring columns of a
    // run, so that a line of a checkpoint's scales (of 2048 columns) is read by one L2
    // instead of eight (2048 x 11008: 112 -> 93 MB, 38.5 -> 37.3 us).
    const uint32_t blocks = gridDim.x * gridDim.y, id = blockIdx.y * gridDim.x + blockIdx.x;
    const uint32_t share = blocks / kXcds, over = blocks % kXcds, xcd = id % kXcds;
    const uint32_t at = xcd * share + (xcd < over ? xcd : over) + id / kXcds;
    const int64_t bx = at % gridDim.x, by = at / gridDim.x;
    const int64_t n0 = bx * kCols;
    const int left = (int)(a.F - n0 < kCols ? a.F - n0 : kCols);
    const Share<1, VEC> sh{left, (int)threadIdx.x % PIECES, PIECES};
    const int64_t last = checkpoint_groups(a.F) - 1;
    int64_t group = (n0 + sh.chunk(0)) / kCheckpointGroup;
    group = group < last ? group : last;
    const int64_t m0 = a.M * by / runs, m1 = a.M * (by + 1) / runs;
    float s[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0][e] = s[1][e] = 0.f;
    for (int64_t m = m0 + r; m < m1; m += kUnroll * kRows) {
        RowRegs<GT, 1, VEC> rg[kUnroll];
        ZRegs<ZT, VEC> rz[kUnroll][2];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {  // rows past the run read its last one
            const int64_t mu = m + u * kRows < m1 ? m + u * kRows : m1 - 1;
            rg[u].load(static_cast<const GT *>(a.grad_y) + mu * a.F + n0, sh);
            rz[u][0].load(a, 2 * mu, n0, sh, group);
            rz[u][1].load(a, 2 * mu + 1, n0, sh, group);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t mu = m + u * kRows;
            if (mu >= m1) break;
            float g[8], z[2][8];
            rg[u].widen(0, sh, g);
            rz[u][0].widen(sh, z[0]);
            rz[u][1].widen(sh, z[1]);
            gated_grads(g, z[0], z[1], a.act);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (a.grad_z) store_share(static_cast<OT *>(a.grad_z) + (2 * mu + h) * a.F + n0, 0, sh, z[h]);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[h][e] += z[h][e];
            }
        }
    }
    if (!a.grad_bias) return;
    const int start = sh.start(0), skip = sh.skip(0);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e >= skip) red[h][r][start + e] = s[h][e];
    __syncthreads();
    float *out = runs == 1 ? a.grad_bias : a.workspace + by * 2 * a.F;
    for (int c = threadIdx.x; c < 2 * kCols; c += kThreads) {
        const int h = c / kCols, n = c % kCols;
        if (n >= left) continue;
        float t = red[h][0][n];
#pragma unroll
        for (int i = 1; i < kRows; ++i) t += red[h][i][n];
        out[h * a.F + n0 + n] = t;
    }
}

// Fewer than eight columns: a thread for each, over a run of rows.
template <typename GT, typename ZT, typename OT>
__global__ __launch_bounds__(64) void gated_grad_few_kernel(const GatedGradArgs a, int64_t runs) {
    const int64_t n = threadIdx.x;
    if (n >= a.F) return;
    const int64_t m0 = a.M * blockIdx.x / runs, m1 = a.M * (blockIdx.x + 1) / runs;
    float s[2] = {0.f, 0.f};
    for (int64_t m = m0; m < m1; ++m) {
        const float g[1] = {Elem<GT>::get(static_cast<const GT *>(a.grad_y), m * a.F + n)};
        float z[2][1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = 2 * m + h;
            if constexpr (sizeof(ZT) == 1) z[h][0] = (float)a.codes[row * a.F + n] * (a.code_scale[row] / 127.0f);
            else z[h][0] = Elem<ZT>::get(static_cast<const ZT *>(a.z), row * a.F + n);
        }
        gated_grads(g, z[0], z[1], a.act);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (a.grad_z) put(static_cast<OT *>(a.grad_z), (2 * m + h) * a.F + n, z[h][0]);
            s[h] += z[h][0];
        }
    }
    if (!a.grad_bias) return;
    float *out = runs == 1 ? a.grad_bias : a.workspace + blockIdx.x * 2 * a.F;
    out[n] = s[0];
    out[a.F + n] = s[1];
}

}  // namespace

int64_t gated_grad_parts(int64_t M, int64_t F) {
    if (M <= kOneRunRows) return 1;
    const int64_t wide = (F + 8 * kWide - 1) / (8 * kWide);
    int64_t runs = (2048 + wide - 1) / wide;  // eight workgroups for each of 256 compute units
    if (runs > (M + 31) / 32) runs = (M + 31) / 32;  // one unrolled step of rows each, at least
    if (runs < (M + kRunRows - 1) / kRunRows) runs = (M + kRunRows - 1) / kRunRows;
    return runs;
}

hipError_t launch_gated_backward(const GatedGradArgs &a, hipStream_t stream) {
    const int64_t runs = gated_grad_parts(a.M, a.F);
    auto run = [&](auto *g, auto *z, auto *o) {
        using GT = Pointee<decltype(g)>;
        using ZT = Pointee<decltype(z)>;
        using OT = Pointee<decltype(o)>;
        auto go = [&](auto pieces_c, auto vec_c) {
            constexpr int P = decltype(pieces_c)::value;
            const dim3 grid((unsigned)((a.F + 8 * P - 1) / (8 * P)), (unsigned)runs);
            hipLaunchKernelGGL((gated_grad_kernel<GT, ZT, OT, P, decltype(vec_c)::value>), grid,
                               dim3(kThreads), 0, stream, a, runs);
            return hipGetLastError();
        };
        auto pieces = [&](auto vec_c) {
            return runs == 1 ? go(std::integral_constant<int, kNarrow>{}, vec_c)
                             : go(std::integral_constant<int, kWide>{}, vec_c);
        };
        hipError_t e;
        if (a.F < 8) {
            hipLaunchKernelGGL((gated_grad_few_kernel<GT, ZT, OT>), dim3((unsigned)runs), dim3(64), 0,
                               stream, a, runs);
            e = hipGetLastError();
        } else {
            e = a.F % 8 == 0 ? pieces(std::true_type{}) : pieces(std::false_type{});
        }
        if (e != hipSuccess || !a.grad_bias || runs == 1) return e;
        return launch_run_sums(a.workspace, a.grad_bias, 2 * a.F, runs, stream);
    };
    return typed(a.gy_dtype, [&](auto g) {
        return typed(a.gz_dtype, [&](auto o) {
            if (!a.z) return run(g, static_cast<int8_t *>(nullptr), o);
            return typed(a.z_dtype, [&](auto z) { return run(g, z, o); });
        });
    });
}

}  // namespace bl
