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
// is written from the same registers.  Bound by HBM: 8192 x 14336 BF16, forward
// with the checkpoint 833 MB in 130 us (6.4 TB/s), without it 591 MB in 87 us (6.8),
// backward from the checkpoint 1182 MB in 177 us (6.7).  To get there each value
// must cost fewer than 38 instructions: packed FP32 products, three-input
// magnitude maxima and, where operands are BF16, the hardware's 2^x and 1/x (with expf and
// an IEEE division the forward took 257 us).
#include "mx_block.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Blocks of a kernel on an SM; the grid is that times the SMs, each warp walks
// the chunks.  Every warp keeps the next chunk's 2 KB (BF16) of loads in flight, so
// two blocks of 16 KB cover HBM's latency: 8192 x 14336 BF16 with the checkpoint
// 130 us at two blocks (<= 128 registers), 153 at three, 258 at four (spills).
// Without the checkpoint a BF16 chunk fits 64 registers: 87 us at four blocks, 92
// at three, 98 at two.
template <int IN, bool KEEP>
constexpr int kForwardBlocks = IN == kBf16 && !KEEP ? 4 : 2;
constexpr int kBackwardBlocks = 2;  // 8192 x 14336 from the checkpoint: 177 us; three 181, four 252 (spills)

// The activation's gate for a pair of values: q, 1 - q, and (GELU) the slope of q's
// argument t = 2z by g.
struct Gate {
    F2 q, rest, inner;
};

// BF16 operands: the hardware's 2^x and 1/x, each within two ulps, on an argument that
// carries the conversion to base 2 in its last constant.  Its rounding moves q by up to
// |t| 2^-24 of its value (4e-6 at -85), far below the 2^-9 of a BF16 result, and 2^x
// overflows to infinity for far negative gates, where q is then 0, as it is below
// 2^-126 (off by less than |g u| 2^-126).
//
// FP32 operands: results keep FP32's precision.  e = exp(-|t|) does not overflow and
// keeps the argument's last bits, 1 / (1 + e) lies in [1/2, 1], and of q and 1 - q the
// smaller is e / (1 + e), without a difference.  It is
// hidden behind HBM but in small calls: SiLU to MXFP8 with checkpoint, 4096 x 14336 FP32
// 96.2 us (95.0 with the other form), 301 x 5120 5.6 (5.1).
template <int ACT, int IN>
__device__ __forceinline__ Gate act_gate(F2 g)
{
    Gate o;
    constexpr bool kFull = IN == kF32;
    constexpr float kTo = kFull ? 1.0f : -1.4426950408889634f;
    F2 t;  // FP32: t; BF16: -t log2(e)
    if (ACT == kActGeluTanh) {
        constexpr float c = 1.5957691216057308f;  // 2 sqrt(2/pi)
        const F2 gg = f2_mul(g, g), k = f2(c * kTo, c * kTo), one = f2(1.0f, 1.0f);
        t = f2_mul(k, f2_mul(g, f2_fma(gg, f2(0.044715f, 0.044715f), one)));
        o.inner = f2_mul(f2(c, c), f2_fma(gg, f2(0.134145f, 0.134145f), one));
    } else {
        t = kFull ? g : f2_mul(g, f2(kTo, kTo));
    }
    float t0, t1, e0, e1, q0, q1;
    f2_split(t, t0, t1);
    if (kFull) {
        e0 = expf(-fabsf(t0));
        e1 = expf(-fabsf(t1));
    } else {
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(t0));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(t1));
    }
    const F2 e = f2(e0, e1);
    f2_split(f2_add(e, f2(1.0f, 1.0f)), e0, e1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q0) : "f"(e0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q1) : "f"(e1));
    const F2 r = f2(q0, q1);
    if (kFull) {
        float s0, s1;
        f2_split(f2_mul(e, r), s0, s1);
        o.q = f2(t0 < 0.0f ? s0 : q0, t1 < 0.0f ? s1 : q1);
        o.rest = f2(t0 < 0.0f ? q0 : s0, t1 < 0.0f ? q1 : s1);
    } else {
        o.q = r;
        o.rest = f2_fma(r, f2(-1.0f, -1.0f), f2(1.0f, 1.0f));
    }
    return o;
}

template <int ACT, int IN, int FMT, bool KEEP>
__global__ void __launch_bounds__(kThreads, kForwardBlocks<IN, KEEP>) glu_kernel(const GluParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t F = p.F;
    ChunkWalk at(F, static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5),
                 static_cast<int64_t>(gridDim.x) * kWarps);
    // the next chunk's loads are in flight while this one is computed
    Raw16<IN> next_g, next_u;
    auto fetch = [&]() {
        const int64_t k = static_cast<int64_t>(at.chunk) * kWarpVals + lane * kLaneVals;
        const bool inside = at.row < p.rows && k < F;
        next_g.load(p.gate + at.row * p.stride + k * E, inside);
        next_u.load(p.up + at.row * p.stride + k * E, inside);
    };
    fetch();
    while (at.row < p.rows) {
        const Raw16<IN> rg = next_g, ru = next_u;
        const int64_t row = at.row, k0 = static_cast<int64_t>(at.chunk) * kWarpVals, k = k0 + lane * kLaneVals;
        const bool inside = k < F;
        at.next();
        fetch();
        float a[kLaneVals];
#pragma unroll
        for (int i = 0; i < kLaneVals / 2; ++i) {
            const F2 g = rg.pair(i);
            f2_split(f2_mul(f2_mul(g, act_gate<ACT, IN>(g).q), ru.pair(i)), a[2 * i], a[2 * i + 1]);
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
            // a row of the checkpoint is two rows of F: the gate's, then the up's (F is a multiple of 32, so no block
            // straddles them)
            const int mode = F % 128 == 0 ? kScaleWords : kScaleBytes;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const Raw16<IN> &x = half ? ru : rg;
                float v[kLaneVals];
#pragma unroll
                for (int i = 0; i < kLaneVals; ++i)
                    v[i] = x.at(i);
                const auto q = mx_encode<kMxfp8>(v, amax_bits(x));
                if (inside)
                    store_codes(p.kept_codes + (2 * row + half) * F, k, q);
                store_scales(p.kept_scales, mode, 2 * row + half, k0, F, lane, q.scode);
            }
        }
    }
    if (FMT != kNoFmt && p.mx.mode == kScaleTiled)
        pad_tiled_scales(p.mx.scales, p.rows, F, static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x,
                         static_cast<int64_t>(gridDim.x) * kThreads);
}

// What a chunk of the backward pass reads.
template <int IN, bool KEPT>
struct BackIn {
    Raw16<IN> dy;
    Raw16<IN> g, u;        // !KEPT
    uint4 qg, qu;          // KEPT
    uint32_t sg, su;

    __device__ __forceinline__ void load(const GluBackParams &p, int64_t row, int64_t k)
    {
        constexpr int E = ElemBytes<IN>::value;
        const bool inside = row < p.rows && k < p.F;
        dy.load(p.dy + row * p.dy_stride + k * E, inside);
        if (KEPT) {
            qg = qu = make_uint4(0, 0, 0, 0);
            sg = su = 127;
            if (inside) {
                const int64_t at = 2 * row * p.F + k;
                qg = __ldcs(reinterpret_cast<const uint4 *>(p.kept_codes + at));
                qu = __ldcs(reinterpret_cast<const uint4 *>(p.kept_codes + at + p.F));
                sg = p.kept_scales[at >> 5];
                su = p.kept_scales[(at + p.F) >> 5];
            }
        } else {
            g.load(p.gate + row * p.stride + k * E, inside);
            u.load(p.up + row * p.stride + k * E, inside);
        }
    }
};

template <int ACT, int IN, int FMT, bool KEPT>
__global__ void __launch_bounds__(kThreads, kBackwardBlocks) glu_backward_kernel(const GluBackParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t F = p.F;
    ChunkWalk at(F, static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5),
                 static_cast<int64_t>(gridDim.x) * kWarps);
    BackIn<IN, KEPT> next;
    next.load(p, at.row, static_cast<int64_t>(at.chunk) * kWarpVals + lane * kLaneVals);
    while (at.row < p.rows) {
        const BackIn<IN, KEPT> in = next;
        const int64_t row = at.row, k0 = static_cast<int64_t>(at.chunk) * kWarpVals, k = k0 + lane * kLaneVals;
        const bool inside = k < F;
        at.next();
        next.load(p, at.row, static_cast<int64_t>(at.chunk) * kWarpVals + lane * kLaneVals);
        F2 g[kLaneVals / 2], u[kLaneVals / 2];
        if (KEPT) {
            decode_e4m3(in.qg, in.sg, g);
            decode_e4m3(in.qu, in.su, u);
        } else {
#pragma unroll
            for (int i = 0; i < kLaneVals / 2; ++i) {
                g[i] = in.g.pair(i);
                u[i] = in.u.pair(i);
            }
        }
        F2 dg2[kLaneVals / 2], du2[kLaneVals / 2], a2[kLaneVals / 2];
#pragma unroll
        for (int i = 0; i < kLaneVals / 2; ++i) {
            const Gate gate = act_gate<ACT, IN>(g[i]);
            const F2 q = gate.q, dy = in.dy.pair(i), f = f2_mul(g[i], q), m = f2_mul(f, gate.rest);
            F2 slope;
            if (ACT == kActSilu) {
                slope = f2_add(m, q);
            } else {
                // where q has reached 0 or 1 the slope is q, also where the inner slope has overflowed
                float m0, m1, s0, s1, q0, q1;
                f2_split(m, m0, m1);
                f2_split(f2_fma(m, gate.inner, q), s0, s1);
                f2_split(q, q0, q1);
                slope = f2(m0 == 0.0f ? q0 : s0, m1 == 0.0f ? q1 : s1);
            }
            dg2[i] = f2_mul(f2_mul(dy, u[i]), slope);
            du2[i] = f2_mul(dy, f);
            a2[i] = f2_mul(f, u[i]);
        }
        float dg[kLaneVals], du[kLaneVals], a[kLaneVals];
        f2_unpack(dg2, dg);
        f2_unpack(du2, du);
        f2_unpack(a2, a);
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
            // Rows of 2F values: the blocks of dup follow those of dgate.  A tile or a word of four scales may hold
            // both where F is not a multiple of 128, so scales go out one byte at a time (words, where they can be,
            // take two shuffles more each: 132 us against 122 at 8192 x 14336 MXFP8).
            if (inside && (lane & 1) == 0) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int64_t kk = k + half * F;
                    const int64_t to = p.mx.mode == kScaleTiled
                                           ? tile_scale_offset(row, kk >> 7, F >> 6) + ((kk >> 5) & 3)
                                           : (2 * row * F + kk) >> 5;
                    p.mx.scales[to] = static_cast<uint8_t>(half ? qu.scode : qg.scode);
                }
            }
        }
    }
    if (FMT != kNoFmt && p.mx.mode == kScaleTiled)
        pad_tiled_scales(p.mx.scales, p.rows, 2 * F, static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x,
                         static_cast<int64_t>(gridDim.x) * kThreads);
}

unsigned row_grid(int64_t rows, int64_t F, int64_t most)
{
    const int64_t chunks = rows * ((F + kWarpVals - 1) / kWarpVals), blocks = (chunks + kWarps - 1) / kWarps;
    return static_cast<unsigned>(blocks < most ? blocks : most);
}

template <int ACT, int IN, int FMT, bool KEEP>
cudaError_t launch_glu_one(const GluParams &p, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg =
        row_launch(row_grid(p.rows, p.F, num_sms * kForwardBlocks<IN, KEEP>), kThreads, 0, s, attr);
    return cudaLaunchKernelEx(&cfg, glu_kernel<ACT, IN, FMT, KEEP>, p);
}

template <int ACT, int IN, int FMT>
cudaError_t launch_glu_keep(const GluParams &p, int num_sms, cudaStream_t s)
{
    return p.kept_codes ? launch_glu_one<ACT, IN, FMT, true>(p, num_sms, s)
                        : launch_glu_one<ACT, IN, FMT, false>(p, num_sms, s);
}

template <int ACT, int IN>
cudaError_t launch_glu_fmt(const GluParams &p, int num_sms, cudaStream_t s)
{
    return p.mx.fmt == kMxfp8   ? launch_glu_keep<ACT, IN, kMxfp8>(p, num_sms, s)
           : p.mx.fmt == kMxfp4 ? launch_glu_keep<ACT, IN, kMxfp4>(p, num_sms, s)
                                : launch_glu_keep<ACT, IN, kNoFmt>(p, num_sms, s);
}

template <int ACT, int IN, int FMT>
cudaError_t launch_back_one(const GluBackParams &p, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = row_launch(row_grid(p.rows, p.F, num_sms * kBackwardBlocks), kThreads, 0, s, attr);
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
