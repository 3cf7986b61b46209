// Backward of the products' extended epilogue:
//   grad_z = grad_y * act'(z),  grad_bias = sum_m grad_z,  grad_residual = res_scale * grad_y.
// act' is recomputed from the stored pre-activation z. grad_bias sums the
// unrounded grad_z. Memory-bound: grad_y and z are read once, grad_z (and
// grad_residual) written once.
#include "activation.hpp"
#include "bl_internal.hpp"
#include "device_util.hpp"

#include <type_traits>

namespace bl {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kChunkRows = 512;  // at most so many terms in one fp32 column sum

template <typename T>
__device__ __forceinline__ void put(T *p, int64_t i, float v) {
    if constexpr (sizeof(T) == 4) p[i] = v;
    else p[i] = (T)f32_to_bf16_rne(v);
}

template <typename GT, typename ZT, typename OT>
__global__ __launch_bounds__(kThreads) void epilogue_grad_kernel(const EpilogueGradArgs a,
                                                                 int64_t parts) {
    const int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (n >= a.N) return;
    const int64_t m0 = a.M * blockIdx.y / parts, m1 = a.M * (blockIdx.y + 1) / parts;
    float s = 0.f;
    for (int64_t m = m0; m < m1; ++m) {
        const int64_t at = m * a.N + n;
        const float g = Elem<GT>::get(static_cast<const GT *>(a.grad_y), at);
        float gz = g;
        if (a.act != kActNone)
            gz = g * activate_grad(Elem<ZT>::get(static_cast<const ZT *>(a.z), at), a.act);
        if (a.grad_z) put(static_cast<OT *>(a.grad_z), at, gz);
        if (a.grad_residual) put(static_cast<GT *>(a.grad_residual), at, a.res_scale * g);
        s += gz;
    }
    if (a.grad_bias) a.workspace[blockIdx.y * a.N + n] = s;
}

__global__ __launch_bounds__(kThreads) void epilogue_grad_sums_kernel(const float *part,
                                                                      float *out, int64_t N,
                                                                      int64_t parts) {
    const int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (n >= N) return;
    double s = 0.0;
    for (int64_t p = 0; p < parts; ++p) s += (double)part[p * N + n];
    out[n] = (float)s;
}

template <typename F>
hipError_t typed(int dtype, F go) {
    return dtype == kF32 ? go(static_cast<float *>(nullptr)) : go(static_cast<uint16_t *>(nullptr));
}
template <typename T> using Pointee = std::remove_pointer_t<T>;

}  // namespace

int64_t epilogue_grad_parts(int64_t M, int64_t N) {
    const int64_t col_blocks = (N + kThreads - 1) / kThreads;
    int64_t p = 2048 / (col_blocks < 1 ? 1 : col_blocks);
    if (p > (M + 15) / 16) p = (M + 15) / 16;
    if (p < (M + kChunkRows - 1) / kChunkRows) p = (M + kChunkRows - 1) / kChunkRows;
    return p < 1 ? 1 : p;
}

hipError_t launch_epilogue_backward(const EpilogueGradArgs &a, hipStream_t stream) {
    const int64_t parts = epilogue_grad_parts(a.M, a.N);
    const unsigned col_blocks = (unsigned)((a.N + kThreads - 1) / kThreads);
    return typed(a.gy_dtype, [&](auto g) {
        return typed(a.z_dtype, [&](auto z) {
            return typed(a.gz_dtype, [&](auto o) {
                using GT = Pointee<decltype(g)>;
                using ZT = Pointee<decltype(z)>;
                using OT = Pointee<decltype(o)>;
                hipLaunchKernelGGL((epilogue_grad_kernel<GT, ZT, OT>),
                                   dim3(col_blocks, (unsigned)parts), dim3(kThreads), 0, stream, a,
                                   parts);
                hipError_t e = hipGetLastError();
                if (e != hipSuccess || !a.grad_bias) return e;
                hipLaunchKernelGGL(epilogue_grad_sums_kernel, dim3(col_blocks), dim3(kThreads), 0,
                                   stream, a.workspace, a.grad_bias, a.N, parts);
                return hipGetLastError();
            });
        });
    });
}

}  // namespace bl
