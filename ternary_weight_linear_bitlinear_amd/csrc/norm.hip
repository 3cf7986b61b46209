// Norms before and after a block, with the block's gate and the residual
// stream between them:
//   p  = norm_post(block)              norm(x) = (x - mu) w / sqrt(var + eps) + bias
//   h' = res_scale * h + gate * p      (RMS: mu = 0, var = mean x^2)
//   n  = norm_pre(h')                  as values, as INT8 codes and scale, or both
// and the backward pass of all of it. Every statistic and sum is held in fp32
// or fp64; h' enters norm_pre unrounded, whatever type it is stored in.
#include "bl_internal.hpp"
#include "device_util.hpp"
#include "row_share.hpp"

namespace bl {
namespace {

constexpr int kThreads = 256;

// Parameter k of a [K] vector, or `none` without one.
template <typename PT>
__device__ __forceinline__ float param(const void *p, int64_t k, float none) {
    return p ? Elem<PT>::get(static_cast<const PT *>(p), k) : none;
}

// Sums of a block's threads, the same value in every thread.
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double red[kThreads / 64];
    v = wave_sum(v);
    __syncthreads();  // the previous sum has been read
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
    __syncthreads();
    double s = red[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) s += red[w];
    return s;
}
__device__ __forceinline__ float block_max(float v) {
    __shared__ float red[kThreads / 64];
    v = wave_max(v);
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
    __syncthreads();
    float m = red[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) m = fmaxf(m, red[w]);
    return m;
}

// ---------------------------------------------------------------------------
// Forward, rows that holds_row() accepts: one workgroup per row, the row held in registers
// from its one read to its one write. Memory-bound: 2048 x 4096 (fp32
// stream, bf16 block, 101 MB) 24 to 26 us, 4 TB/s, against 5.1 TB/s for a 1 GiB copy (19 us
// where the outputs stay in the caches); 8192 rows 76 us, 5.3 TB/s. Codes in place of
// values 23.6 us (92 MB), values, codes and statistics 28.7 us (109 MB). 2048 x 11008
// 60 us, 2048 x 16384 84 us, 1024 x 32768 99 us (four chunks: 4.1 TB/s). One row of 4096
// takes 2.9 us, which is latency.
//
// Thread t owns J chunks of eight consecutive elements (chunks t, t + T, ...;
// row_share.hpp). Every load of the row is issued before the first reduction. A
// statistic is a sum in fp32 over at most 8 J elements of a thread, a wave's 64
// lanes and 16 waves, so at most 8 J + 10 additions follow one another.
constexpr int kMaxWaves = 16;
constexpr int64_t kRegElems = 8 * 64 * kMaxWaves;  // of a row, for each chunk per thread
// Chunks per thread: the fewest threads that hold the row wait least on one
// another, the most finish a single row soonest. From two rows per compute unit on
// rows of 2048 elements and more take two chunks. Their time against one chunk's (RMS, bf16
// block, with an fp32 and with a bf16 stream, more data than the caches hold):
//   width     333 rows   512        1024       2048       8192
//   2048     +15 +17%   +14 +17%    +5  +3%     0  +1%    +5  +1%
//   4096      +3  +5%    +5  +6%    -3  -2%    +5  -2%     0  -8%
//   5001      +2  -3%    +6  -2%   -14 -31%    -4 -21%   -11 -26%
//   6144       0  -2%    +6  +3%    +1  -8%    +2  -4%    -6 -13%
//   8192     -10 -17%   -11  -7%   -12 -16%   -12 -23%   -17 -29%
// (8192 x 8192 bf16 144.5 -> 101.9 us, 512 x 2048 4.6 -> 5.4 us.) The narrow end of the
// rule costs up to 0.8 us a call; rows of 8192 would gain from 257 rows on.
// Rows of more than 16384 elements take four chunks, which with an fp32 block
// spill 8 to 53 registers (1024 x 32768 118 us, 4.5 TB/s).
constexpr int64_t kManyRows = 512;
inline bool holds_row(int64_t K) { return K >= 8 && K <= 4 * kRegElems; }

// Reductions over the workgroup. Each wave leaves its value in `red`, which is
// this reduction's own, so one barrier is enough; then every thread reads all of
// them, four to a load and all loads at once (one by one, the LDS latency
// of up to 16 waves' values cost more than the rest of the reduction). Entries of
// absent waves are zero (clear_absent(), before the first barrier).
__device__ __forceinline__ void clear_absent(float *red, int slots, int waves) {
    for (int i = threadIdx.x; i < slots * kMaxWaves; i += blockDim.x)
        if (i % kMaxWaves >= waves) red[i] = 0.f;
}
template <typename OP>
__device__ __forceinline__ float across_waves(const float *red, int waves, OP op) {
    const float4 *q = reinterpret_cast<const float4 *>(red);
    auto of = [&](const float4 &a) { return op(op(a.x, a.y), op(a.z, a.w)); };
    if (waves <= 4) return of(q[0]);
    if (waves <= 8) {
        const float4 a = q[0], b = q[1];
        return op(of(a), of(b));
    }
    const float4 a = q[0], b = q[1], c = q[2], d = q[3];
    return op(op(of(a), of(b)), op(of(c), of(d)));
}
__device__ __forceinline__ float group_sum(float v, float *red, int waves) {
    v = wave_sum_dpp(v);
    if (waves == 1) return v;
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
    lds_barrier();
    return across_waves(red, waves, [](float a, float b) { return a + b; });
}
// The same of one value for each of a thread's J chunks, added in the order in which
// workgroups of J times the threads would add one each, so that a row's result
// does not depend on how many rows go with it. (Rows of more chunks than 16 waves hold
// always take the same J, and their threads add their own first.)
template <int J>
__device__ __forceinline__ float group_sum_chunks(const float (&v)[J], float *red, int waves) {
    if constexpr (J == 1) {
        return group_sum(v[0], red, waves);
    } else {
        if (J * waves > kMaxWaves) {
            float t = v[0];
#pragma unroll
            for (int j = 1; j < J; ++j) t += v[j];
            return group_sum(t, red, waves);
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const float t = wave_sum_dpp(v[j]);
            if (threadIdx.x % 64 == 0) red[j * waves + threadIdx.x / 64] = t;
        }
        lds_barrier();
        return across_waves(red, J * waves, [](float a, float b) { return a + b; });
    }
}
// Two sums at once; red: 2 kMaxWaves entries.
__device__ __forceinline__ float2 group_sum2(float v, float w, float *red, int waves) {
    v = wave_sum_dpp(v);
    w = wave_sum_dpp(w);
    if (waves == 1) return make_float2(v, w);
    if (threadIdx.x % 64 == 0) {
        red[threadIdx.x / 64] = v;
        red[kMaxWaves + threadIdx.x / 64] = w;
    }
    lds_barrier();
    auto add = [](float a, float b) { return a + b; };
    return make_float2(across_waves(red, waves, add), across_waves(red + kMaxWaves, waves, add));
}
__device__ __forceinline__ float group_max0(float v, float *red, int waves) {  // of values >= 0
    v = wave_max0_dpp(v);
    if (waves == 1) return v;
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
    lds_barrier();
    return across_waves(red, waves, [](float a, float b) { return fmaxf(a, b); });
}

// Chunk j of a [K] parameter vector in fp32, ones without the vector.
template <typename PT, int J, bool VEC>
__device__ __forceinline__ void load_param(const void *p, int j, const Share<J, VEC> &sh, float (&w)[8]) {
    if (!p) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
        return;
    }
    Raw8<PT> r;
    load_chunk(static_cast<const PT *>(p), j, sh, r);
    r.widen(w);
}
// The same times a second vector.
template <typename PT, int J, bool VEC>
__device__ __forceinline__ void load_params(const void *p, const void *q, int j,
                                            const Share<J, VEC> &sh, float (&w)[8]) {
    load_param<PT>(p, j, sh, w);
    if (!q) return;
    float f[8];
    load_param<PT>(q, j, sh, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= f[e];
}

template <typename HT, typename XT, typename PT, int J, bool VEC>
__global__ __launch_bounds__(64 * kMaxWaves) void block_norm_kernel(const BlockNormArgs a,
                                                                    int64_t m0) {
    __shared__ __attribute__((aligned(16))) float red[5][kMaxWaves];
    const int64_t m = m0 + blockIdx.x, K = a.K;
    const int waves = blockDim.x / 64;
    clear_absent(red[0], 4, J * waves > kMaxWaves ? waves : J * waves);  // sums
    clear_absent(red[4], 1, waves);                                      // the maximum
    const Share<J, VEC> sh{(int)K, (int)threadIdx.x, (int)blockDim.x};
    const float inv_k = 1.0f / (float)K;
    const bool block = a.block != nullptr, token = a.gate_kind == kGateToken;
    const void *gc = a.gate_kind == kGateChannel ? a.gate : nullptr;

    RowRegs<XT, J, VEC> rb, rg;
    RowRegs<HT, J, VEC> rh;
    if (block) rb.load(static_cast<const XT *>(a.block) + m * K, sh);
    rh.load(static_cast<const HT *>(a.h) + m * K, sh);
    if (token) rg.load(static_cast<const XT *>(a.gate) + m * K, sh);
    // norm_post's weight and a gate per channel act as one factor. With one
    // chunk per thread the parameters are fetched along with the row; with more
    // they would spill, and come (from L2) where they are used.
    constexpr bool kEarly = J == 1;
    float wp[8], wn[8], pb[8], nb[8];
    if constexpr (kEarly) {
        load_params<PT>(a.post.weight, gc, 0, sh, wp);
        load_param<PT>(a.pre.weight, 0, sh, wn);
        if (a.post.bias) load_params<PT>(a.post.bias, gc, 0, sh, pb);
        if (a.pre.bias) load_param<PT>(a.pre.bias, 0, sh, nb);
    }

    // mean and 1 / deviation of the share x (zero past K)
    auto stats_of = [&](const NormSide &s, const float (&x)[J][8], float *red0, float *red1, float &mean,
                        float &rstd) {
        mean = 0.f;
        rstd = 1.f;
        if (s.kind == kNormNone) return;
        float t[J];
        if (s.kind == kNormLayer) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                t[j] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) t[j] += x[j][e];
            }
            mean = group_sum_chunks(t, red0, waves) * inv_k;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float d[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = x[j][e] - mean;
            if (s.kind == kNormLayer) clear_past(j, sh, d);
            t[j] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) t[j] = __builtin_fmaf(d[e], d[e], t[j]);
        }
        rstd = 1.0f / sqrtf(group_sum_chunks(t, red1, waves) * inv_k + s.eps);
    };

    float v[J][8];  // h'
    float mean_b = 0.f, rstd_b = 1.f, mean_h, rstd_h;
#pragma unroll
    for (int j = 0; j < J; ++j) rh.widen(j, sh, v[j]);
    if (block) {
        float b[J][8];
#pragma unroll
        for (int j = 0; j < J; ++j) rb.widen(j, sh, b[j]);
        stats_of(a.post, b, red[0], red[1], mean_b, rstd_b);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if constexpr (!kEarly) load_params<PT>(a.post.weight, gc, j, sh, wp);
#pragma unroll
            for (int e = 0; e < 8; ++e) b[j][e] = (b[j][e] - mean_b) * wp[e] * rstd_b;
            if (a.post.bias) {
                if constexpr (!kEarly) load_params<PT>(a.post.bias, gc, j, sh, pb);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[j][e] += pb[e];
            }
            if (token) {
                float g[8];
                rg.widen(j, sh, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[j][e] *= g[e];
            }
        }
        HT *out = static_cast<HT *>(a.h_out) + m * K;
#pragma unroll
        for (int j = 0; j < J; ++j) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = __builtin_fmaf(a.res_scale, v[j][e], b[j][e]);
            clear_past(j, sh, v[j]);
            store_share(out, j, sh, v[j]);
        }
    }
    stats_of(a.pre, v, red[2], red[3], mean_h, rstd_h);
    if (a.stats && threadIdx.x == 0)
        reinterpret_cast<float4 *>(a.stats)[m] = make_float4(mean_b, rstd_b, mean_h, rstd_h);
    if (a.pre.kind == kNormNone) return;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if constexpr (!kEarly) load_param<PT>(a.pre.weight, j, sh, wn);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = (v[j][e] - mean_h) * wn[e] * rstd_h;
        if (a.pre.bias) {
            if constexpr (!kEarly) load_param<PT>(a.pre.bias, j, sh, nb);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] += nb[e];
        }
    }
    if (a.n) {
        XT *out = static_cast<XT *>(a.n) + m * K;
#pragma unroll
        for (int j = 0; j < J; ++j) store_share(out, j, sh, v[j]);
    }
    if (a.xq) {
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            clear_past(j, sh, v[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[j][e]));
        }
        const float s = fmaxf(group_max0(top, red[4], waves), 1e-6f);
        const float y = 1.0f / s;
        if (threadIdx.x == 0) a.scale[m] = s;
        int8_t *out = a.xq + m * K;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            int8_t *p = out + sh.start(j);
            const int skip = sh.skip(j);
            if (skip == 0) {
                const uint32_t lo = quant4(v[j][0], v[j][1], v[j][2], v[j][3], s, y);
                const uint32_t hi = quant4(v[j][4], v[j][5], v[j][6], v[j][7], s, y);
                if constexpr (VEC) *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
                else *reinterpret_cast<Bytes8 *>(p) = Bytes8{{lo, hi}};
            } else if constexpr (!VEC) {
#pragma unroll
                for (int e = 1; e < 8; ++e)
                    if (e >= skip) p[e] = quant1(v[j][e], s, y);
            }
        }
    }
}

// Other rows: one row per workgroup, any K: each statistic is a pass over the row (which
// stays in the caches), the last pass writes. Every element is read and written
// by one thread, and nothing is written before the last pass, so h_out may be h.
// 512 x 40000 387 us, 0.6 TB/s; one row of 40000 171 us: single elements by 256 threads,
// four waves a row. Usual hidden widths lie between these rows' (under 8, over 32768).
template <typename HT, typename XT, typename PT>
__global__ __launch_bounds__(kThreads) void block_norm_rows_kernel(const BlockNormArgs a,
                                                                   int64_t m0) {
    const int64_t m = m0 + blockIdx.x, K = a.K;
    const HT *h = static_cast<const HT *>(a.h) + m * K;
    const XT *b = a.block ? static_cast<const XT *>(a.block) + m * K : nullptr;
    const XT *gt = a.gate_kind == kGateToken ? static_cast<const XT *>(a.gate) + m * K : nullptr;
    const void *gc = a.gate_kind == kGateChannel ? a.gate : nullptr;

    auto stats_of = [&](const NormSide &s, auto get, float &mean, float &rstd) {
        mean = 0.f;
        rstd = 1.f;
        if (s.kind == kNormNone) return;
        if (s.kind == kNormLayer) {
            double t = 0.0;
            for (int64_t k = threadIdx.x; k < K; k += kThreads) t += (double)get(k);
            mean = (float)(block_sum(t) / (double)K);
        }
        double v = 0.0;
        for (int64_t k = threadIdx.x; k < K; k += kThreads) {
            const double d = (double)get(k) - (double)mean;
            v += d * d;
        }
        rstd = 1.0f / sqrtf((float)(block_sum(v) / (double)K) + s.eps);
    };
    auto apply = [&](const NormSide &s, float x, int64_t k, float mean, float rstd) {
        if (s.kind == kNormNone) return x;
        const float t = (x - mean) * param<PT>(s.weight, k, 1.f) * rstd;
        return s.bias ? t + param<PT>(s.bias, k, 0.f) : t;
    };

    float mean_b = 0.f, rstd_b = 1.f, mean_h, rstd_h;
    if (b) stats_of(a.post, [&](int64_t k) { return Elem<XT>::get(b, k); }, mean_b, rstd_b);
    auto stream = [&](int64_t k) {  // h'
        const float hv = Elem<HT>::get(h, k);
        if (!b) return hv;
        float p = apply(a.post, Elem<XT>::get(b, k), k, mean_b, rstd_b);
        if (gt) p *= Elem<XT>::get(gt, k);
        if (gc) p *= param<PT>(gc, k, 1.f);
        return __builtin_fmaf(a.res_scale, hv, p);
    };
    stats_of(a.pre, stream, mean_h, rstd_h);
    float s = 1.f, y = 1.f;
    if (a.xq) {
        float top = 0.f;
        for (int64_t k = threadIdx.x; k < K; k += kThreads)
            top = fmaxf(top, fabsf(apply(a.pre, stream(k), k, mean_h, rstd_h)));
        s = fmaxf(block_max(top), 1e-6f);
        y = 1.0f / s;
    }
    if (threadIdx.x == 0) {
        if (a.xq) a.scale[m] = s;
        if (a.stats)
            reinterpret_cast<float4 *>(a.stats)[m] = make_float4(mean_b, rstd_b, mean_h, rstd_h);
    }
    for (int64_t k = threadIdx.x; k < K; k += kThreads) {
        const float hv = stream(k);
        if (a.h_out) put(static_cast<HT *>(a.h_out), m * K + k, hv);
        const float nv = apply(a.pre, hv, k, mean_h, rstd_h);
        if (a.n) put(static_cast<XT *>(a.n), m * K + k, nv);
        if (a.xq) a.xq[m * K + k] = quant1(nv, s, y);
    }
}

// ---------------------------------------------------------------------------
// Backward. With x^ = (x - mu) rs and v the gradient of a norm's output, the
// gradient of its input is rs (w v - mean(w v) - x^ mean(w v x^)), the first
// mean for LayerNorm only. Rows first:
//   d = grad_h' + J_pre^T grad_n;  grad_h = res_scale d;  grad_block = J_post^T (gate d)
// then the columns: sum_m of grad_n x^_pre, grad_n, (d g) x^_post and d g (g: a
// gate per token, else 1); a gate per channel factors out of its sums.
//
// Rows that grad_holds_row() accepts take both in one kernel: a workgroup walks
// a run of rows, each held in registers (one or two chunks of eight elements
// per thread), with the next row's loads in flight while the current one is
// reduced, and keeps its columns' sums in registers. The sums of a run (at most
// kChunkRows rows) are fp32; block_norm_grad_sums_kernel adds the runs in fp64,
// in a fixed order. 256 runs of 512 threads do best: with more, the partial sums
// and the lost overlap cost more than the extra waves give (8192 x 4096: 128 runs
// 179 us, 256 138 us, 512 143 us, 1024 151 us; 4096 x 4096 fp32 stream and grad_n,
// 335 MB, 70 us, 4.8 TB/s, and 5 us for the sums).
// Rows of two chunks spill: up to 65 registers without biases, 26 to 185 with them (four
// column sums of two chunks are 64 registers beside two rows). 2048 x 8192, the
// sums included: RMS 90.6 us (3.7 TB/s), LayerNorm with biases 124 us (2.7), fp32
// throughout 119 and 175 us, bf16 throughout 56 and 75 us.
constexpr int64_t kChunkRows = 512;
constexpr int kGradThreads = 512;  // at most: two waves of 256 registers per SIMD
inline bool grad_holds_row(int64_t K) { return K >= 8 && K <= 2 * 8 * kGradThreads; }

template <typename HT, typename XT, typename NT, typename PT, int J, bool BIAS, bool VEC>
__global__ __launch_bounds__(kGradThreads) void block_norm_grad_kernel(const BlockNormGradArgs a,
                                                                       int64_t runs, bool cols) {
    using S = Share<J, VEC>;
    __shared__ __attribute__((aligned(16))) float red[2][2][2 * kMaxWaves];  // [row parity][norm]
    const int64_t K = a.K;
    const int waves = blockDim.x / 64;
    clear_absent(red[0][0], 8, waves);
    const S sh{(int)K, (int)threadIdx.x, (int)blockDim.x};
    const float inv_k = 1.0f / (float)K;
    const bool has_g = a.grad_h_out != nullptr, has_n = a.grad_n != nullptr;
    const bool block = a.block != nullptr, token = a.gate_kind == kGateToken;
    const bool post = a.post.kind != kNormNone;
    const void *gc = a.gate_kind == kGateChannel ? a.gate : nullptr;
    const int64_t m0 = a.M * blockIdx.x / runs, m1 = a.M * (blockIdx.x + 1) / runs;

    // norm_pre's weight, norm_post's times a gate per channel, and (for the gradient
    // of a gate per token) norm_post's bias. What the registers cannot hold lies in
    // LDS, each thread's own: read from memory in the loop, it would be waited for
    // together with the next row's loads, which are issued before it
    // (2048 x 8192, fp32 stream and grad_n, 100.1 -> 88.8 us).
    extern __shared__ float4 own[];
    constexpr int kBiasSlot = 0, kPreSlot = 1, kPostSlot = 2;
    auto keep = [&](int slot, int j, const float (&w)[8]) {
        float4 *q = own + (slot * J + j) * 2 * blockDim.x + threadIdx.x;
        q[0] = make_float4(w[0], w[1], w[2], w[3]);
        q[blockDim.x] = make_float4(w[4], w[5], w[6], w[7]);
    };
    auto fetch = [&](int slot, int j, float (&w)[8]) {
        const float4 *q = own + (slot * J + j) * 2 * blockDim.x + threadIdx.x;
        const float4 lo = q[0], hi = q[blockDim.x];
        w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w;
        w[4] = hi.x; w[5] = hi.y; w[6] = hi.z; w[7] = hi.w;
    };
    const bool gate_bias = token && a.grad_gate && a.post.bias;
    float wn[8], wp[8];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        load_param<PT>(a.pre.weight, j, sh, wn);
        load_params<PT>(a.post.weight, gc, j, sh, wp);
        if constexpr (J > 1) {
            keep(kPreSlot, j, wn);
            keep(kPostSlot, j, wp);
        }
        if (gate_bias) {
            float pb[8];
            load_param<PT>(a.post.bias, j, sh, pb);
            keep(kBiasSlot, j, pb);
        }
    }
    constexpr int kSums = BIAS ? 4 : 2;
    float acc[kSums][J][8];
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[i][j][e] = 0.f;

    RowRegs<HT, J, VEC> rG, rh;
    RowRegs<NT, J, VEC> rn;
    RowRegs<XT, J, VEC> rb, rg;
    float4 st_next;
    auto load_row = [&](int64_t m) {
        const int64_t at = m * K;
        if (has_g) rG.load(static_cast<const HT *>(a.grad_h_out) + at, sh);
        if (has_n) rn.load(static_cast<const NT *>(a.grad_n) + at, sh);
        rh.load(static_cast<const HT *>(a.h_out) + at, sh);
        if (block) rb.load(static_cast<const XT *>(a.block) + at, sh);
        if (token) rg.load(static_cast<const XT *>(a.gate) + at, sh);
        st_next = reinterpret_cast<const float4 *>(a.stats)[m];
    };
    if (m0 < m1) load_row(m0);
    for (int64_t m = m0; m < m1; ++m) {
        float d[J][8], g[J][8], hat[J][8], b[J][8], gt[J][8];
        const float4 st = st_next;
#pragma unroll
        for (int j = 0; j < J; ++j) {
#pragma unroll
            for (int e = 0; e < 8; ++e) d[j][e] = g[j][e] = b[j][e] = 0.f, gt[j][e] = 1.f;
            if (has_g) rG.widen(j, sh, d[j]);
            if (has_n) rn.widen(j, sh, g[j]);
            rh.widen(j, sh, hat[j]);
            if (block) rb.widen(j, sh, b[j]);
            if (token) rg.widen(j, sh, gt[j]);
        }
        if (m + 1 < m1) load_row(m + 1);
        const int p = m & 1;

        if (has_n) {
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if constexpr (J > 1) fetch(kPreSlot, j, wn);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    hat[j][e] = (hat[j][e] - st.z) * st.w;
                    const float wv = g[j][e] * wn[e];
                    acc[0][j][e] = __builtin_fmaf(g[j][e], hat[j][e], acc[0][j][e]);
                    if constexpr (BIAS) acc[2][j][e] += g[j][e];
                    g[j][e] = wv;
                    s1 += wv;
                    s2 = __builtin_fmaf(wv, hat[j][e], s2);
                }
            }
            const float2 c = group_sum2(s1, s2, red[p][0], waves);
            const float c1 = a.pre.kind == kNormLayer ? c.x * inv_k : 0.f, c2 = c.y * inv_k;
#pragma unroll
            for (int j = 0; j < J; ++j) {
#pragma unroll
                for (int e = 0; e < 8; ++e) d[j][e] += st.w * (g[j][e] - c1 - hat[j][e] * c2);
                clear_past(j, sh, d[j]);
            }
        }
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float out[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) out[e] = block ? a.res_scale * d[j][e] : d[j][e];
            store_share(static_cast<HT *>(a.grad_h) + m * K, j, sh, out);
            if (!block) continue;
            if constexpr (J > 1) fetch(kPostSlot, j, wp);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = d[j][e] * gt[j][e];
                b[j][e] = (b[j][e] - st.x) * st.y;  // x^ of norm_post (b itself without it)
                gt[j][e] = v * wp[e];
                s1 += gt[j][e];
                s2 = __builtin_fmaf(gt[j][e], b[j][e], s2);
                acc[1][j][e] = __builtin_fmaf(v, b[j][e], acc[1][j][e]);
                if constexpr (BIAS) acc[3][j][e] += v;
            }
            if (token && a.grad_gate) {
                float pb[8];
                if (gate_bias) fetch(kBiasSlot, j, pb);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float pv = b[j][e] * wp[e];
                    out[e] = d[j][e] * (gate_bias ? pv + pb[e] : pv);
                }
                store_share(static_cast<XT *>(a.grad_gate) + m * K, j, sh, out);
            }
        }
        if (!block) continue;
        float e1 = 0.f, e2 = 0.f;
        if (post) {
            const float2 c = group_sum2(s1, s2, red[p][1], waves);
            e1 = a.post.kind == kNormLayer ? c.x * inv_k : 0.f;
            e2 = c.y * inv_k;
        }
        if (!a.grad_block) continue;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (post) {
#pragma unroll
                for (int e = 0; e < 8; ++e) gt[j][e] = st.y * (gt[j][e] - e1 - b[j][e] * e2);
            }
            store_share(static_cast<XT *>(a.grad_block) + m * K, j, sh, gt[j]);
        }
    }
    if (!cols) return;
    float *part = a.workspace + (int64_t)blockIdx.x * kSums * K;
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) store_share(part + i * K, j, sh, acc[i][j]);
}

// Sums of the runs' partials [runs][sums][K], in fp64: 32 columns of one sum per
// workgroup, the runs split over its 32 rows of threads (of the 256 runs of a
// full card each thread has eight loads, all in flight at once).
constexpr int kSumRows = 32;
// Order of the sums: grad_n x^_pre, (d g) x^_post, grad_n, d g.
template <typename PT>
__global__ __launch_bounds__(32 * kSumRows) void block_norm_grad_sums_kernel(
    const BlockNormGradArgs a, const float *parts, int64_t runs, int sums) {
    __shared__ double red[2][kSumRows][33];
    const int c = threadIdx.x % 32, r = threadIdx.x / 32, y = blockIdx.y;
    const int64_t k = (int64_t)blockIdx.x * 32 + c, stride = sums * a.K;
    const bool biased = sums > 2;
    double s1 = 0.0, s0 = 0.0;  // of norm_pre (y = 0) or norm_post (y = 1)
    if (k < a.K) {
        const float *p1 = parts + y * a.K + k, *p0 = p1 + 2 * a.K;
#pragma unroll 8
        for (int64_t i = r; i < runs; i += kSumRows) {
            s1 += (double)p1[i * stride];
            if (biased) s0 += (double)p0[i * stride];
        }
    }
    red[0][r][c] = s1;
    red[1][r][c] = s0;
    __syncthreads();
    // two rows of threads finish: 0 the first sum, 1 the second
    if (r < 2) {
        double s = 0.0;
        if (r == 0 || biased) {
#pragma unroll
            for (int i = 0; i < kSumRows; ++i) s += red[r][i][c];
        }
        red[r][0][c] = s;
    }
    __syncthreads();
    if (r > 0 || k >= a.K) return;
    s1 = red[0][0][c];
    s0 = red[1][0][c];
    if (y == 0) {
        if (a.grad_pre_weight) a.grad_pre_weight[k] = (float)s1;
        if (a.grad_pre_bias) a.grad_pre_bias[k] = (float)s0;
        return;
    }
    const bool gc = a.gate_kind == kGateChannel;
    const double g = gc ? (double)param<PT>(a.gate, k, 1.f) : 1.0;
    if (a.grad_post_weight) a.grad_post_weight[k] = (float)(g * s1);
    if (a.grad_post_bias) a.grad_post_bias[k] = (float)(g * s0);
    if (gc && a.grad_gate)
        static_cast<float *>(a.grad_gate)[k] = (float)((double)param<PT>(a.post.weight, k, 1.f) * s1 +
                                                       (double)param<PT>(a.post.bias, k, 0.f) * s0);
}

// Other rows: a workgroup per row with a pass per statistic, then the columns
// in a kernel of their own that forms d again. Single elements, and every input
// walked several times: 2048 x 11008 453 us, 2048 x 16384 686 us (1 TB/s of what
// must move).
template <typename HT, typename XT, typename NT, typename PT>
struct GradRow {
    const BlockNormGradArgs &a;
    const HT *G, *h;
    const NT *gn;
    const XT *b, *gt;
    float4 st;
    __device__ GradRow(const BlockNormGradArgs &a_, int64_t m) : a(a_) {
        const int64_t at = m * a.K;
        G = a.grad_h_out ? static_cast<const HT *>(a.grad_h_out) + at : nullptr;
        h = static_cast<const HT *>(a.h_out) + at;
        gn = a.grad_n ? static_cast<const NT *>(a.grad_n) + at : nullptr;
        b = a.block ? static_cast<const XT *>(a.block) + at : nullptr;
        gt = a.gate_kind == kGateToken ? static_cast<const XT *>(a.gate) + at : nullptr;
        st = reinterpret_cast<const float4 *>(a.stats)[m];
    }
    __device__ float grad_n(int64_t k) const { return Elem<NT>::get(gn, k); }
    __device__ float pre_hat(int64_t k) const { return (Elem<HT>::get(h, k) - st.z) * st.w; }
    __device__ float post_hat(int64_t k) const { return (Elem<XT>::get(b, k) - st.x) * st.y; }
    __device__ float d(int64_t k, float c1, float c2) const {
        float v = G ? Elem<HT>::get(G, k) : 0.f;
        if (gn) {
            const float wv = grad_n(k) * param<PT>(a.pre.weight, k, 1.f);
            v += st.w * (wv - c1 - pre_hat(k) * c2);
        }
        return v;
    }
    __device__ float gated(float dv, int64_t k) const { return gt ? dv * Elem<XT>::get(gt, k) : dv; }
};

template <typename HT, typename XT, typename NT, typename PT>
__global__ __launch_bounds__(kThreads) void block_norm_grad_rows_kernel(const BlockNormGradArgs a,
                                                                        int64_t m0) {
    const int64_t m = m0 + blockIdx.x, K = a.K;
    const GradRow<HT, XT, NT, PT> r(a, m);
    const void *gc = a.gate_kind == kGateChannel ? a.gate : nullptr;
    float c1 = 0.f, c2 = 0.f, e1 = 0.f, e2 = 0.f;
    if (r.gn) {
        double s1 = 0.0, s2 = 0.0;
        for (int64_t k = threadIdx.x; k < K; k += kThreads) {
            const float wv = r.grad_n(k) * param<PT>(a.pre.weight, k, 1.f);
            s1 += (double)wv;
            s2 += (double)wv * (double)r.pre_hat(k);
        }
        if (a.pre.kind == kNormLayer) c1 = (float)(block_sum(s1) / (double)K);
        c2 = (float)(block_sum(s2) / (double)K);
    }
    if (threadIdx.x == 0)
        reinterpret_cast<float2 *>(a.workspace)[m] = make_float2(c1, c2);
    auto into_post = [&](float dv, int64_t k) {  // gradient of norm_post's output, times its weight
        float u = r.gated(dv, k) * param<PT>(a.post.weight, k, 1.f);
        return gc ? u * param<PT>(gc, k, 1.f) : u;
    };
    if (r.b && a.post.kind != kNormNone) {
        double s1 = 0.0, s2 = 0.0;
        for (int64_t k = threadIdx.x; k < K; k += kThreads) {
            const float u = into_post(r.d(k, c1, c2), k);
            s1 += (double)u;
            s2 += (double)u * (double)r.post_hat(k);
        }
        if (a.post.kind == kNormLayer) e1 = (float)(block_sum(s1) / (double)K);
        e2 = (float)(block_sum(s2) / (double)K);
    }
    for (int64_t k = threadIdx.x; k < K; k += kThreads) {
        const float dv = r.d(k, c1, c2);
        put(static_cast<HT *>(a.grad_h), m * K + k, r.b ? a.res_scale * dv : dv);
        if (!r.b) continue;
        const float u = into_post(dv, k);
        const float hat = r.post_hat(k);
        if (a.grad_block)
            put(static_cast<XT *>(a.grad_block), m * K + k,
                a.post.kind != kNormNone ? r.st.y * (u - e1 - hat * e2) : u);
        if (r.gt && a.grad_gate) {
            const float p = hat * param<PT>(a.post.weight, k, 1.f) + param<PT>(a.post.bias, k, 0.f);
            put(static_cast<XT *>(a.grad_gate), m * K + k, dv * p);
        }
    }
}

// Column sums over the rows of one chunk, in fp32: at most kChunkRows terms,
// the chunks are then added in fp64 (block_norm_grad_sums_kernel).
constexpr int kAllSums = 4;
int64_t grad_chunks(int64_t M, int64_t K) {
    const int64_t col_blocks = (K + kThreads - 1) / kThreads;
    int64_t p = 2048 / col_blocks;  // about eight workgroups for each compute unit
    if (p > (M + 15) / 16) p = (M + 15) / 16;
    if (p < (M + kChunkRows - 1) / kChunkRows) p = (M + kChunkRows - 1) / kChunkRows;
    return p < 1 ? 1 : p;
}

template <typename HT, typename XT, typename NT, typename PT>
__global__ __launch_bounds__(kThreads) void block_norm_grad_cols_kernel(const BlockNormGradArgs a,
                                                                        int64_t chunks) {
    const int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (k >= a.K) return;
    const int64_t m0 = a.M * blockIdx.y / chunks, m1 = a.M * (blockIdx.y + 1) / chunks;
    float s[kAllSums] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t m = m0; m < m1; ++m) {
        const GradRow<HT, XT, NT, PT> r(a, m);
        const float2 c = reinterpret_cast<const float2 *>(a.workspace)[m];
        if (r.gn) {
            const float g = r.grad_n(k);
            s[0] = __builtin_fmaf(g, r.pre_hat(k), s[0]);
            s[2] += g;
        }
        if (r.b) {
            const float v = r.gated(r.d(k, c.x, c.y), k);
            s[1] = __builtin_fmaf(v, r.post_hat(k), s[1]);
            s[3] += v;
        }
    }
    float *out = a.workspace + 2 * a.M + (int64_t)blockIdx.y * kAllSums * a.K + k;
#pragma unroll
    for (int i = 0; i < kAllSums; ++i) out[i * a.K] = s[i];
}

// Threads of the fused kernel, and its runs of rows: as many workgroups as keep
// kGradThreads threads on each of 256 compute units, at most kChunkRows rows each.
int64_t grad_threads(int64_t K) {
    const int64_t chunks = (K + 7) / 8;
    return ((K <= 8 * kGradThreads ? chunks : (chunks + 1) / 2) + 63) / 64 * 64;
}
int64_t grad_runs(int64_t M, int64_t K) {
    int64_t r = 256 * (kGradThreads / grad_threads(K));
    if (r > M) r = M;
    if (r < (M + kChunkRows - 1) / kChunkRows) r = (M + kChunkRows - 1) / kChunkRows;
    return r;
}

}  // namespace

namespace {
// One workgroup per row: launches of at most this many rows, since a grid holds
// fewer than 2^32 threads in a dimension. launch(first row, rows).
constexpr int64_t kLaunchRows = 1 << 21;
template <typename F>
hipError_t by_rows(int64_t M, F launch) {
    for (int64_t m0 = 0; m0 < M; m0 += kLaunchRows) {
        launch(m0, dim3((unsigned)(M - m0 < kLaunchRows ? M - m0 : kLaunchRows)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}
}  // namespace

hipError_t launch_block_norm(const BlockNormArgs &a, hipStream_t stream) {
    return typed(a.h_dtype, [&](auto h) {
        return typed(a.x_dtype, [&](auto x) {
            return typed(a.p_dtype, [&](auto p) {
                using HT = Pointee<decltype(h)>;
                using XT = Pointee<decltype(x)>;
                using PT = Pointee<decltype(p)>;
                if (!holds_row(a.K))
                    return by_rows(a.M, [&](int64_t m0, dim3 grid) {
                        hipLaunchKernelGGL((block_norm_rows_kernel<HT, XT, PT>), grid,
                                           dim3(kThreads), 0, stream, a, m0);
                    });
                auto go = [&](auto j_c, auto vec_c) {
                    constexpr int J = decltype(j_c)::value;
                    const int64_t threads = ((a.K + 8 * J - 1) / (8 * J) + 63) / 64 * 64;
                    return by_rows(a.M, [&](int64_t m0, dim3 grid) {
                        hipLaunchKernelGGL((block_norm_kernel<HT, XT, PT, J, decltype(vec_c)::value>),
                                           grid, dim3((unsigned)threads), 0, stream, a, m0);
                    });
                };
                auto chunks = [&](auto vec_c) {
                    if (a.K <= kRegElems && !(a.M >= kManyRows && a.K >= 2048))
                        return go(std::integral_constant<int, 1>{}, vec_c);
                    if (a.K <= 2 * kRegElems) return go(std::integral_constant<int, 2>{}, vec_c);
                    return go(std::integral_constant<int, 4>{}, vec_c);
                };
                return a.K % 8 == 0 ? chunks(std::true_type{}) : chunks(std::false_type{});
            });
        });
    });
}

int64_t block_norm_grad_workspace(int64_t M, int64_t K) {
    if (grad_holds_row(K)) return grad_runs(M, K) * kAllSums * K;
    return 2 * M + grad_chunks(M, K) * kAllSums * K;
}

hipError_t launch_block_norm_backward(const BlockNormGradArgs &a, hipStream_t stream) {
    const bool cols = a.grad_pre_weight || a.grad_pre_bias || a.grad_post_weight ||
                      a.grad_post_bias || (a.grad_gate && a.gate_kind == kGateChannel);
    // sums of grad_n and d g: for bias gradients, and for a channel gate's over a bias
    const bool bias = a.grad_pre_bias || a.grad_post_bias ||
                      (a.grad_gate && a.gate_kind == kGateChannel && a.post.bias);
    const int64_t runs = grad_holds_row(a.K) ? grad_runs(a.M, a.K) : grad_chunks(a.M, a.K);
    hipError_t e = typed(a.h_dtype, [&](auto h) {
        return typed(a.x_dtype, [&](auto x) {
            return typed(a.gn_dtype, [&](auto n) {
                return typed(a.p_dtype, [&](auto p) {
                    using HT = Pointee<decltype(h)>;
                    using XT = Pointee<decltype(x)>;
                    using NT = Pointee<decltype(n)>;
                    using PT = Pointee<decltype(p)>;
                    if (grad_holds_row(a.K)) {
                        auto go = [&](auto j_c, auto bias_c, auto vec_c) {
                            constexpr int J = decltype(j_c)::value;
                            auto kern = block_norm_grad_kernel<HT, XT, NT, PT, J, decltype(bias_c)::value,
                                                               decltype(vec_c)::value>;
                            const int64_t threads = grad_threads(a.K);
                            // 32 bytes a thread and chunk: one slot, three with two chunks
                            const size_t lds = (size_t)threads * 32 * (J > 1 ? 3 * J : 1);
                            static LdsFlag raised;
                            hipError_t e = allow_dynamic_lds(kern, J > 1 ? kGradThreads * 192 : lds, &raised);
                            if (e != hipSuccess) return e;
                            hipLaunchKernelGGL(kern, dim3((unsigned)runs), dim3((unsigned)threads), lds,
                                               stream, a, runs, cols);
                            return hipGetLastError();
                        };
                        auto biased = [&](auto j_c, auto vec_c) {
                            return bias ? go(j_c, std::true_type{}, vec_c) : go(j_c, std::false_type{}, vec_c);
                        };
                        const std::integral_constant<int, 1> one;
                        const std::integral_constant<int, 2> two;
                        auto chunks = [&](auto vec_c) {
                            return a.K <= 8 * kGradThreads ? biased(one, vec_c) : biased(two, vec_c);
                        };
                        return a.K % 8 == 0 ? chunks(std::true_type{}) : chunks(std::false_type{});
                    }
                    hipError_t e = by_rows(a.M, [&](int64_t m0, dim3 grid) {
                        hipLaunchKernelGGL((block_norm_grad_rows_kernel<HT, XT, NT, PT>), grid,
                                           dim3(kThreads), 0, stream, a, m0);
                    });
                    if (e != hipSuccess || !cols) return e;
                    hipLaunchKernelGGL((block_norm_grad_cols_kernel<HT, XT, NT, PT>),
                                       dim3((unsigned)((a.K + kThreads - 1) / kThreads), (unsigned)runs),
                                       dim3(kThreads), 0, stream, a, runs);
                    return hipGetLastError();
                });
            });
        });
    });
    if (e != hipSuccess || !cols) return e;
    const bool fused = grad_holds_row(a.K);
    const float *parts = a.workspace + (fused ? 0 : 2 * a.M);
    const int sums = fused && !bias ? 2 : kAllSums;
    const dim3 grid((unsigned)((a.K + 31) / 32), 2);
    return typed(a.p_dtype, [&](auto p) {
        hipLaunchKernelGGL((block_norm_grad_sums_kernel<Pointee<decltype(p)>>), grid,
                           dim3(32 * kSumRows), 0, stream, a, parts, runs, sums);
        return hipGetLastError();
    });
}

}  // namespace bl
