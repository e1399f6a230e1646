// glu.cu -- gated activation a = act(g) * u with an MX output and an MXFP8
// checkpoint of its inputs, and its gradient from that checkpoint.
//
//   SiLU:      act(g) = g * q,  q = 1 / (1 + exp(-g))
//   tanh-GELU: act(g) = g * q,  q = (1 + tanh(z)) / 2 = 1 / (1 + exp(-2z)),  z = sqrt(2/pi) (g + 0.044715 g^3)
//   act'(g) = q + g * q * (1 - q) * t',  t' = 1 (SiLU) or 2 dz/dg (GELU)
//   dg = dy * u * act'(g),  du = dy * act(g)
//
// Elementwise over rows apart from the scale blocks: a warp takes 512
// consecutive values of a row, every byte of input is read once and every output
// is written from the same registers.
#include "mx_block.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// act(g) and its slope's parts share q; expf overflows to infinity for very
// negative arguments, where q is then 0 and the products are the limits.
template <int ACT>
__device__ __forceinline__ float act_gate(float g, float &inner)
{
    float t = g;
    inner = 1.0f;
    if (ACT == kActGeluTanh) {
        const float c = 1.5957691216057308f;  // 2 sqrt(2/pi)
        t = c * fmaf(0.044715f * g * g, g, g);
        inner = c * fmaf(0.134145f * g, g, 1.0f);
    }
    return 1.0f / (1.0f + expf(-t));
}

template <int ACT, int IN, int FMT, bool KEEP>
__global__ void __launch_bounds__(kThreads) glu_kernel(const GluParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t F = p.F, per_row = (F + kWarpVals - 1) / kWarpVals, units = p.rows * per_row;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
         u += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t row = u / per_row, k0 = (u - row * per_row) * kWarpVals, k = k0 + lane * kLaneVals;
        const bool inside = k < F;
        Raw16<IN> rg, ru;
        rg.load(p.gate + row * p.stride + k * E, inside);
        ru.load(p.up + row * p.stride + k * E, inside);
        float a[kLaneVals];
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i) {
            float inner;
            const float g = rg.at(i);
            a[i] = g * act_gate<ACT>(g, inner) * ru.at(i);
        }
        if (p.y && inside)
            store16<IN>(p.y + (row * F + k) * E, a);
        if (FMT != kNoFmt) {
            const auto q = mx_encode<FMT == kNoFmt ? kMxfp8 : FMT>(a);
            if (inside)
                store_codes(p.mx.codes + row * (FMT == kMxfp8 ? F : F >> 1), k, q);
            store_scales(p.mx.scales, p.mx.mode, row, k0, F, lane, q.scode);
        }
        if (KEEP) {
            // gate in the first F columns, up in the last F; F is a multiple of 32, so a block never straddles
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float v[kLaneVals];
#pragma unroll
                for (int i = 0; i < kLaneVals; ++i)
                    v[i] = half ? ru.at(i) : rg.at(i);
                const auto q = mx_encode<kMxfp8>(v);
                if (inside) {
                    store_codes(p.kept_codes + (2 * row + half) * F, k, q);
                    if ((lane & 1) == 0)
                        p.kept_scales[((2 * row + half) * F + k) >> 5] = static_cast<uint8_t>(q.scode);
                }
            }
        }
    }
    if (FMT != kNoFmt && p.mx.mode == kScaleTiled)
        pad_tiled_scales(p.mx.scales, p.rows, F, static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x,
                         static_cast<int64_t>(gridDim.x) * kThreads);
}

template <int ACT, int IN, int FMT, bool KEPT>
__global__ void __launch_bounds__(kThreads) glu_backward_kernel(const GluBackParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t F = p.F, per_row = (F + kWarpVals - 1) / kWarpVals, units = p.rows * per_row;
    for (int64_t n = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); n < units;
         n += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t row = n / per_row, k0 = (n - row * per_row) * kWarpVals, k = k0 + lane * kLaneVals;
        const bool inside = k < F;
        Raw16<IN> rdy;
        rdy.load(p.dy + row * p.dy_stride + k * E, inside);
        float g[kLaneVals], u[kLaneVals];
        if (KEPT) {
            uint4 qg = make_uint4(0, 0, 0, 0), qu = qg;
            uint32_t sg = 127, su = 127;
            if (inside) {
                const int64_t at = 2 * row * F + k;
                qg = __ldcs(reinterpret_cast<const uint4 *>(p.kept_codes + at));
                qu = __ldcs(reinterpret_cast<const uint4 *>(p.kept_codes + at + F));
                sg = p.kept_scales[at >> 5];
                su = p.kept_scales[(at + F) >> 5];
            }
            decode_e4m3(qg, sg, g);
            decode_e4m3(qu, su, u);
        } else {
            Raw16<IN> rg, ru;
            rg.load(p.gate + row * p.stride + k * E, inside);
            ru.load(p.up + row * p.stride + k * E, inside);
#pragma unroll
            for (int i = 0; i < kLaneVals; ++i) {
                g[i] = rg.at(i);
                u[i] = ru.at(i);
            }
        }
        float dg[kLaneVals], du[kLaneVals], a[kLaneVals];
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i) {
            float inner;
            const float q = act_gate<ACT>(g[i], inner), dy = rdy.at(i), f = g[i] * q;
            // where q has reached 0 or 1 the slope is q, also where `inner` has overflowed
            const float m = f * (1.0f - q);
            dg[i] = dy * u[i] * (m == 0.0f ? q : fmaf(m, inner, q));
            du[i] = dy * f;
            a[i] = f * u[i];
        }
        if (p.a && inside)
            store16<IN>(p.a + (row * F + k) * E, a);
        if (p.dgu && inside) {
            store16<IN>(p.dgu + (2 * row * F + k) * E, dg);
            store16<IN>(p.dgu + ((2 * row + 1) * F + k) * E, du);
        }
        if (FMT != kNoFmt) {
            const auto qg = mx_encode<FMT == kNoFmt ? kMxfp8 : FMT>(dg);
            const auto qu = mx_encode<FMT == kNoFmt ? kMxfp8 : FMT>(du);
            uint8_t *codes = p.mx.codes + 2 * row * (FMT == kMxfp8 ? F : F >> 1);
            if (inside) {
                store_codes(codes, k, qg);
                store_codes(codes, F + k, qu);
            }
            // rows of 2F values: the blocks of dup follow those of dgate.  A tile or a word of four scales may hold
            // both where F is not a multiple of 128, so scales go out one byte at a time.
            if (inside && (lane & 1) == 0) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int64_t kk = k + half * F;
                    const int64_t at = p.mx.mode == kScaleTiled
                                           ? tile_scale_offset(row, kk >> 7, F >> 6) + ((kk >> 5) & 3)
                                           : (2 * row * F + half * F + k) >> 5;
                    p.mx.scales[at] = static_cast<uint8_t>(half ? qu.scode : qg.scode);
                }
            }
        }
    }
    if (FMT != kNoFmt && p.mx.mode == kScaleTiled)
        pad_tiled_scales(p.mx.scales, p.rows, 2 * F, static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x,
                         static_cast<int64_t>(gridDim.x) * kThreads);
}

unsigned row_grid(int64_t rows, int64_t F, int num_sms)
{
    const int64_t units = rows * ((F + kWarpVals - 1) / kWarpVals);
    const int64_t blocks = (units + kWarps - 1) / kWarps, cap = static_cast<int64_t>(num_sms) * 8;
    return static_cast<unsigned>(blocks < cap ? blocks : cap);
}

template <int ACT, int IN, int FMT>
cudaError_t launch_glu_one(const GluParams &p, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = row_launch(row_grid(p.rows, p.F, num_sms), kThreads, 0, s, attr);
    return p.kept_codes ? cudaLaunchKernelEx(&cfg, glu_kernel<ACT, IN, FMT, true>, p)
                        : cudaLaunchKernelEx(&cfg, glu_kernel<ACT, IN, FMT, false>, p);
}

template <int ACT, int IN>
cudaError_t launch_glu_fmt(const GluParams &p, int num_sms, cudaStream_t s)
{
    return p.mx.fmt == kMxfp8   ? launch_glu_one<ACT, IN, kMxfp8>(p, num_sms, s)
           : p.mx.fmt == kMxfp4 ? launch_glu_one<ACT, IN, kMxfp4>(p, num_sms, s)
                                : launch_glu_one<ACT, IN, kNoFmt>(p, num_sms, s);
}

template <int ACT, int IN, int FMT>
cudaError_t launch_back_one(const GluBackParams &p, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = row_launch(row_grid(p.rows, p.F, num_sms), kThreads, 0, s, attr);
    return p.kept_codes ? cudaLaunchKernelEx(&cfg, glu_backward_kernel<ACT, IN, FMT, true>, p)
                        : cudaLaunchKernelEx(&cfg, glu_backward_kernel<ACT, IN, FMT, false>, p);
}

template <int ACT, int IN>
cudaError_t launch_back_fmt(const GluBackParams &p, int num_sms, cudaStream_t s)
{
    return p.mx.fmt == kMxfp8   ? launch_back_one<ACT, IN, kMxfp8>(p, num_sms, s)
           : p.mx.fmt == kMxfp4 ? launch_back_one<ACT, IN, kMxfp4>(p, num_sms, s)
                                : launch_back_one<ACT, IN, kNoFmt>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_glu(const GluParams &p, int act, int in_dtype, int num_sms, cudaStream_t s)
{
    if (act == kActSilu)
        return in_dtype == kBf16 ? launch_glu_fmt<kActSilu, kBf16>(p, num_sms, s)
                                 : launch_glu_fmt<kActSilu, kF32>(p, num_sms, s);
    return in_dtype == kBf16 ? launch_glu_fmt<kActGeluTanh, kBf16>(p, num_sms, s)
                             : launch_glu_fmt<kActGeluTanh, kF32>(p, num_sms, s);
}

cudaError_t launch_glu_backward(const GluBackParams &p, int act, int in_dtype, int num_sms, cudaStream_t s)
{
    if (act == kActSilu)
        return in_dtype == kBf16 ? launch_back_fmt<kActSilu, kBf16>(p, num_sms, s)
                                 : launch_back_fmt<kActSilu, kF32>(p, num_sms, s);
    return in_dtype == kBf16 ? launch_back_fmt<kActGeluTanh, kBf16>(p, num_sms, s)
                             : launch_back_fmt<kActGeluTanh, kF32>(p, num_sms, s);
}

}  // namespace mxg
