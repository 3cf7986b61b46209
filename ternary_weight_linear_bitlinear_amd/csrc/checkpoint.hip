// Activations kept in 8 bits between the forward and the backward pass. The
// quantiser is that of the activations ([b158] §3.2, §5.2), over groups of 64
// columns of a row instead of the whole row:
//   s = max(max |x|, 1e-6),  q = clamp(round(x / s * 127), -127, 127)
// and a kept value stands for q * s / 127, within s / 254 of x but for four fp32 roundings
// (of x / s, its product with 127, s / 127 and its product with q: 2^-22 s). Memory-bound: x is
// read once, 1 + 4 / 64 bytes written for each element; restoring is the reverse.
//
// Eight threads hold a group, eight columns each, and take its maximum across
// lanes. A workgroup covers W pieces of eight columns (W = 8 .. 256, a power of two)
// and 256 / W rows at a time, four of them in flight. 2048 x 11008 in bf16: 13.2 us, 69 MB,
// 5.3 TB/s; restored 11.7 us (the codes are still cached); 333 x 5001 in fp32 4.5 and 5.1 us.
#include "bl_internal.hpp"
#include "device_util.hpp"
#include "row_share.hpp"

namespace bl {
namespace {

constexpr int kThreads = 256, kUnroll = 4;

struct KeptArgs {
    const void *x;  // restored from: codes
    int8_t *codes;
    float *scale;
    void *y;  // restored to
    int64_t M, K;
    int wide;  // log2 of W
};

// This thread's piece of eight columns and rows.
template <bool VEC>
struct KeptShare {
    Share<1, VEC> sh;
    int64_t n0, row0, step, group, groups;
    __device__ __forceinline__ explicit KeptShare(const KeptArgs &a) {
        const int W = 1 << a.wide, piece = threadIdx.x & (W - 1);
        n0 = (int64_t)blockIdx.y * 8 * W;
        const int64_t left = a.K - n0;
        sh = Share<1, VEC>{(int)(left < 8 * W ? left : 8 * W), piece, W};
        step = kThreads >> a.wide;
        row0 = (int64_t)blockIdx.x * kUnroll * step + (threadIdx.x >> a.wide);
        groups = checkpoint_groups(a.K);
        group = (n0 + 8 * piece) / kCheckpointGroup;  // (past the last one: nothing is owned)
    }
};

template <typename XT, bool VEC>
__global__ __launch_bounds__(kThreads) void checkpoint_kernel(const KeptArgs a) {
    const KeptShare<VEC> k(a);
    RowRegs<XT, 1, VEC> rx[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {  // rows past the last read it again
        const int64_t m = k.row0 + u * k.step < a.M ? k.row0 + u * k.step : a.M - 1;
        rx[u].load(static_cast<const XT *>(a.x) + m * a.K + k.n0, k.sh);
    }
    const int start = k.sh.start(0), skip = k.sh.skip(0);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t m = k.row0 + u * k.step;
        float v[8], top = 0.f;
        rx[u].widen(0, k.sh, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
        const float s = fmaxf(max8_dpp(top), 1e-6f), r = 1.0f / s;
        if (m >= a.M || skip >= 8) continue;
        const uint32_t q[2] = {quant4(v[0], v[1], v[2], v[3], s, r), quant4(v[4], v[5], v[6], v[7], s, r)};
        int8_t *p = a.codes + m * a.K + k.n0 + start;
        if (skip == 0) {
            if constexpr (VEC) *reinterpret_cast<uint2 *>(p) = make_uint2(q[0], q[1]);
            else *reinterpret_cast<Bytes8 *>(p) = Bytes8{{q[0], q[1]}};
        } else {
#pragma unroll
            for (int e = 1; e < 8; ++e)
                if (e >= skip) p[e] = (int8_t)(q[e / 4] >> (8 * (e % 4)));
        }
        if (threadIdx.x % 8 == 0) a.scale[m * k.groups + k.group] = s;
    }
}

template <typename YT, bool VEC>
__global__ __launch_bounds__(kThreads) void checkpoint_restore_kernel(const KeptArgs a) {
    const KeptShare<VEC> k(a);
    const int64_t group = k.group < k.groups ? k.group : k.groups - 1;
    Kept8 rx[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t m = k.row0 + u * k.step < a.M ? k.row0 + u * k.step : a.M - 1;
        load_kept(static_cast<const int8_t *>(a.x) + m * a.K + k.n0, a.scale + m * k.groups, group, k.sh, rx[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t m = k.row0 + u * k.step;
        if (m >= a.M) continue;
        float v[8];
        rx[u].widen(v);
        store_share(static_cast<YT *>(a.y) + m * a.K + k.n0, 0, k.sh, v);
    }
}

// Rows of fewer than eight columns: one group, a thread for each row.
template <typename XT>
__global__ __launch_bounds__(kThreads) void checkpoint_few_kernel(const KeptArgs a) {
    const int64_t m = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (m >= a.M) return;
    const XT *x = static_cast<const XT *>(a.x) + m * a.K;
    float s = 1e-6f;
    for (int k = 0; k < (int)a.K; ++k) s = fmaxf(s, fabsf(Elem<XT>::get(x, k)));
    for (int k = 0; k < (int)a.K; ++k) a.codes[m * a.K + k] = quant1(Elem<XT>::get(x, k), s, 1.0f / s);
    a.scale[m] = s;
}
template <typename YT>
__global__ __launch_bounds__(kThreads) void checkpoint_restore_few_kernel(const KeptArgs a) {
    const int64_t m = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (m >= a.M) return;
    const float f = a.scale[m] / 127.0f;
    for (int k = 0; k < (int)a.K; ++k)
        put(static_cast<YT *>(a.y), m * a.K + k, (float)static_cast<const int8_t *>(a.x)[m * a.K + k] * f);
}

// W: as many pieces side by side as waste the fewest lanes past a row's last group,
// 32 at least where the row has them (512 bytes of bf16); 256 for rows so long that
// the grid's second dimension could run out.
int wide_of(int64_t K) {
    const int64_t pieces = 8 * checkpoint_groups(K);
    if (pieces >= 65536) return 8;
    int best = 3;
    while (best < 5 && (1 << best) < pieces) ++best;
    int64_t cost = INT64_MAX;
    for (int w = best; w <= 8; ++w) {
        const int64_t c = ((pieces + (1 << w) - 1) >> w) << w;
        if (c <= cost) cost = c, best = w;
    }
    return best;
}
dim3 kept_grid(const KeptArgs &a) {
    const int64_t W = 1 << a.wide, rows = kUnroll * (kThreads >> a.wide);
    return dim3((unsigned)((a.M + rows - 1) / rows),
                (unsigned)((8 * checkpoint_groups(a.K) + W - 1) >> a.wide));
}
dim3 few_grid(const KeptArgs &a) { return dim3((unsigned)((a.M + kThreads - 1) / kThreads)); }

}  // namespace

hipError_t launch_checkpoint(const void *x, int x_dtype, int64_t M, int64_t K, int8_t *codes,
                             float *scale, hipStream_t stream) {
    const KeptArgs a{x, codes, scale, nullptr, M, K, wide_of(K)};
    return typed(x_dtype, [&](auto t) {
        using XT = Pointee<decltype(t)>;
        if (K < 8)
            hipLaunchKernelGGL(checkpoint_few_kernel<XT>, few_grid(a), dim3(kThreads), 0, stream, a);
        else if (K % 8 == 0)
            hipLaunchKernelGGL((checkpoint_kernel<XT, true>), kept_grid(a), dim3(kThreads), 0, stream, a);
        else
            hipLaunchKernelGGL((checkpoint_kernel<XT, false>), kept_grid(a), dim3(kThreads), 0, stream, a);
        return hipGetLastError();
    });
}

hipError_t launch_checkpoint_restore(const int8_t *codes, const float *scale, int64_t M, int64_t K,
                                     void *y, int y_dtype, hipStream_t stream) {
    const KeptArgs a{codes, nullptr, const_cast<float *>(scale), y, M, K, wide_of(K)};
    return typed(y_dtype, [&](auto t) {
        using YT = Pointee<decltype(t)>;
        if (K < 8)
            hipLaunchKernelGGL(checkpoint_restore_few_kernel<YT>, few_grid(a), dim3(kThreads), 0, stream, a);
        else if (K % 8 == 0)
            hipLaunchKernelGGL((checkpoint_restore_kernel<YT, true>), kept_grid(a), dim3(kThreads), 0, stream, a);
        else
            hipLaunchKernelGGL((checkpoint_restore_kernel<YT, false>), kept_grid(a), dim3(kThreads), 0, stream, a);
        return hipGetLastError();
    });
}

}  // namespace bl
