// norm.cu -- RMS norm with the residual's addition and an MX output, and its
// gradient.
//
//   h = x + r;  rstd = 1/sqrt(mean(h^2) + eps);  y = h * rstd * w
//   p = dy * w;  dx = rstd * p - h * rstd^3 * mean(p * h) + dh;  dw = sum_rows dy * h * rstd
//
// Both are one pass over rows that never leave the registers between their
// reduction and their use: the forward reads x (and r) once and writes h, y,
// codes and scales from the same registers, in FP32 until the final rounding.
#include "mx_block.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kMaxThreads = 512;

// Sum of v over the block; `part` holds one float per warp.  One barrier: a
// caller that sums again passes the other of two buffers.
__device__ __forceinline__ float block_sum(float v, float *part)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
    v = warp_sum(v);
    if (lane == 0)
        part[warp] = v;
    __syncthreads();
    v = lane < nwarps ? part[lane] : 0.0f;
    return warp_sum(v);
}

// ------------------------------------------------------------------ forward --
// One block per row, a thread holds NCH runs of 16 values.
template <int IN, int WT, int FMT, int NCH>
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_kernel(const NormParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    __shared__ float part[32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int64_t row = blockIdx.x, K = p.K;
    const char *xrow = p.x + row * p.x_stride;
    const char *rrow = p.residual ? p.residual + row * p.residual_stride : nullptr;

    Raw16<IN> x[NCH], r[NCH];
    Raw16<WT> w[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int64_t k = (c * nwarps + warp) * kWarpVals + lane * kLaneVals;
        x[c].load(xrow + k * E, k < K);
        r[c].load(rrow + k * E, k < K && rrow != nullptr);
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int64_t k = (c * nwarps + warp) * kWarpVals + lane * kLaneVals;
        w[c].load(p.weight + k * ElemBytes<WT>::value, k < K);
    }
    float h[NCH][kLaneVals];
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i) {
            h[c][i] = rrow ? x[c].at(i) + r[c].at(i) : x[c].at(i);
            ss = fmaf(h[c][i], h[c][i], ss);
        }
    const float rstd = __frsqrt_rn(block_sum(ss, part) / static_cast<float>(K) + p.eps);
    if (threadIdx.x == 0 && p.rstd)
        p.rstd[row] = rstd;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int64_t k0 = (c * nwarps + warp) * kWarpVals;
        const int64_t k = k0 + lane * kLaneVals;
        const bool inside = k < K;
        if (p.h && inside)
            store16<IN>(p.h + (row * K + k) * E, h[c]);
        float y[kLaneVals];
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i)
            y[i] = h[c][i] * rstd * w[c].at(i);
        if (p.y && inside)
            store16<IN>(p.y + (row * K + k) * E, y);
        if (FMT != kNoFmt) {
            const auto q = mx_encode<FMT == kNoFmt ? kMxfp8 : FMT>(y);
            if (inside)
                store_codes(p.mx.codes + row * (FMT == kMxfp8 ? K : K >> 1), k, q);
            store_scales(p.mx.scales, p.mx.mode, row, k0, K, lane, q.scode);
        }
    }
    if (FMT != kNoFmt && p.mx.mode == kScaleTiled)
        pad_tiled_scales(p.mx.scales, p.rows, K, row * blockDim.x + threadIdx.x,
                         static_cast<int64_t>(gridDim.x) * blockDim.x);
}

// ----------------------------------------------------------------- backward --
// Blocks stride over the rows; a thread keeps its columns' share of dw in
// registers and leaves it in partial[block].
template <int IN, int WT, int NCH>
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_backward_kernel(const NormBackParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    __shared__ float part[2][32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int64_t K = p.K;
    float dw[NCH][kLaneVals];
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i)
            dw[c][i] = 0.0f;
    int flip = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= 1) {
        Raw16<IN> dy[NCH], h[NCH], dh[NCH];
        Raw16<WT> w[NCH];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int64_t k = (c * nwarps + warp) * kWarpVals + lane * kLaneVals;
            dy[c].load(p.dy + row * p.dy_stride + k * E, k < K);
            h[c].load(p.h + row * p.h_stride + k * E, k < K);
            dh[c].load(p.dh + row * p.dh_stride + k * E, k < K && p.dh != nullptr);
            w[c].load(p.weight + k * ElemBytes<WT>::value, k < K);
        }
        const float rstd = p.rstd[row];
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int i = 0; i < kLaneVals; ++i)
                dot = fmaf(dy[c].at(i) * w[c].at(i), h[c].at(i), dot);
        dot = block_sum(dot, part[flip]);
        const float coef = rstd * rstd * rstd * (dot / static_cast<float>(K));
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int64_t k = (c * nwarps + warp) * kWarpVals + lane * kLaneVals;
            float dx[kLaneVals];
#pragma unroll
            for (int i = 0; i < kLaneVals; ++i) {
                const float g = dy[c].at(i), v = h[c].at(i);
                dx[i] = fmaf(-v, coef, rstd * (g * w[c].at(i))) + dh[c].at(i);
                dw[c][i] = fmaf(g, v * rstd, dw[c][i]);
            }
            if (k < K)
                store16<IN>(p.dx + (row * K + k) * E, dx);
        }
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int64_t k = (c * nwarps + warp) * kWarpVals + lane * kLaneVals;
        if (k < K)
            store16<kF32>(reinterpret_cast<char *>(p.partial + blockIdx.x * K + k), dw[c]);
    }
}

// dw[k] = sum of partial[b][k] over the blocks, in block order within each of
// eight slices and then over the slices: the same sum every run.
__global__ void __launch_bounds__(256) rmsnorm_dweight_kernel(const float *partial, int blocks, int64_t K, float *dw)
{
    __shared__ float part[8][32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t k = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float v = 0.0f;
#pragma unroll 4
    for (int b = slice; b < blocks; b += 8)
        v += partial[b * K + k];
    part[slice][lane] = v;
    __syncthreads();
    if (slice == 0) {
#pragma unroll
        for (int s = 1; s < 8; ++s)
            v += part[s][lane];
        dw[k] = v;
    }
}

struct Shape {
    int nch, threads;
};

Shape pick_shape(int64_t K)
{
    Shape s;
    s.nch = K <= 8192 ? 1 : K <= 16384 ? 2 : 4;
    const int64_t warps = (K + s.nch * kWarpVals - 1) / (s.nch * kWarpVals);
    s.threads = static_cast<int>(warps) * 32;
    return s;
}

template <int IN, int WT, int FMT>
cudaError_t launch_forward(const NormParams &p, cudaStream_t s)
{
    const Shape sh = pick_shape(p.K);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = row_launch(static_cast<unsigned>(p.rows), sh.threads, 0, s, attr);
    return sh.nch == 1   ? cudaLaunchKernelEx(&cfg, rmsnorm_kernel<IN, WT, FMT, 1>, p)
           : sh.nch == 2 ? cudaLaunchKernelEx(&cfg, rmsnorm_kernel<IN, WT, FMT, 2>, p)
                         : cudaLaunchKernelEx(&cfg, rmsnorm_kernel<IN, WT, FMT, 4>, p);
}

template <int IN, int WT>
cudaError_t launch_forward_fmt(const NormParams &p, cudaStream_t s)
{
    return p.mx.fmt == kMxfp8   ? launch_forward<IN, WT, kMxfp8>(p, s)
           : p.mx.fmt == kMxfp4 ? launch_forward<IN, WT, kMxfp4>(p, s)
                                : launch_forward<IN, WT, kNoFmt>(p, s);
}

template <int IN, int WT>
cudaError_t launch_backward(const NormBackParams &p, int num_sms, cudaStream_t s)
{
    const Shape sh = pick_shape(p.K);
    int64_t blocks = 2 * num_sms;
    blocks = blocks < kNormBackBlocks ? blocks : kNormBackBlocks;
    blocks = blocks < p.rows ? blocks : p.rows;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = row_launch(static_cast<unsigned>(blocks), sh.threads, 0, s, attr);
    const cudaError_t e = sh.nch == 1   ? cudaLaunchKernelEx(&cfg, rmsnorm_backward_kernel<IN, WT, 1>, p)
                          : sh.nch == 2 ? cudaLaunchKernelEx(&cfg, rmsnorm_backward_kernel<IN, WT, 2>, p)
                                        : cudaLaunchKernelEx(&cfg, rmsnorm_backward_kernel<IN, WT, 4>, p);
    if (e != cudaSuccess)
        return e;
    const cudaLaunchConfig_t cfg2 = row_launch(static_cast<unsigned>(p.K / 32), 256, 0, s, attr);
    return cudaLaunchKernelEx(&cfg2, rmsnorm_dweight_kernel, static_cast<const float *>(p.partial),
                              static_cast<int>(blocks), p.K, p.dweight);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormParams &p, int in_dtype, int weight_dtype, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    if (in_dtype == kBf16)
        return weight_dtype == kBf16 ? launch_forward_fmt<kBf16, kBf16>(p, s) : launch_forward_fmt<kBf16, kF32>(p, s);
    return weight_dtype == kBf16 ? launch_forward_fmt<kF32, kBf16>(p, s) : launch_forward_fmt<kF32, kF32>(p, s);
}

cudaError_t launch_rmsnorm_backward(const NormBackParams &p, int in_dtype, int weight_dtype, int num_sms,
                                    cudaStream_t s)
{
    if (in_dtype == kBf16)
        return weight_dtype == kBf16 ? launch_backward<kBf16, kBf16>(p, num_sms, s)
                                     : launch_backward<kBf16, kF32>(p, num_sms, s);
    return weight_dtype == kBf16 ? launch_backward<kF32, kBf16>(p, num_sms, s)
                                 : launch_backward<kF32, kF32>(p, num_sms, s);
}

}  // namespace mxg
