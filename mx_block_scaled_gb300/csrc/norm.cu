// norm.cu -- RMS norm with the residual's addition and an MX output, and its
// gradient.
//
//   h = x + r;  rstd = 1/sqrt(mean(h^2) + eps);  y = h * rstd * w
//   p = dy * w;  n = h * rstd;  dx = rstd * (p - n * mean(p * n)) + dh;  dw = sum_rows dy * n
//
// (mean(p * n) is taken as rstd * mean(p * h), one factor a row.  No power of rstd is
// formed: rstd^3 leaves FP32 for rows of 1e13 or 1e-13, which n and the factor do not.)
//
// Both are one pass over the rows, bound by HBM.  The forward keeps a row in the
// registers of one block between its reduction and its use and writes h, y, codes
// and scales from them, in FP32 until the final rounding; blocks on the same SM
// cover each other's reductions: 16384 x 8192 BF16 with residual and tiled MXFP8
// (944 MB) 135 us, 7.0 TB/s.  The backward also sums over rows, so its blocks stay
// and hide the reduction in a pipeline instead: 16384 x 8192 BF16 (1074 MB) 175 us,
// 6.1 TB/s, 8192 x 4096 (268 MB) 51 us, of which 4 are the second launch.
#include "mx_block.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kMaxThreads = 512;

// Many narrow rows (up to 1024 values): rows side by side in blocks of four warps, since
// a multiprocessor takes up small blocks too slowly (16384 x 384: 10.2 us, 17.0 with a
// block a row; 16384 x 608 without a residual 11.6 and 17.1).  Wider rows gain nothing
// (16384 x 2016 without a residual 21.7 us against 19.8), nor do fewer (2048 x 512: 3.2
// against 3.0).
constexpr int64_t kSideK = 1024, kSideRows = 4096;
constexpr int kSideThreads = 128;

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
// A block takes a row, a thread NCH runs of 16 values of it.  Sums and products are
// packed pairs: at 3 bytes a value (BF16 to MXFP8 without a residual) a value may cost
// 17 instructions before they bind instead of HBM.  The weight is kept in L1 for the
// SM's next rows: fetched from L2 for every row, its few lines hold up all SMs (8192 x
// 2016 FP32: 32 us, 46 without; 1504: 24 and 38).  SIDE: blockDim.y rows beside each
// other.
template <int IN, int WT, int FMT, int NCH, bool RES, bool SIDE>
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_kernel(const NormParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    __shared__ float part[32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int64_t row = SIDE ? static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y : blockIdx.x, K = p.K;
    const int part0 = SIDE ? threadIdx.y * nwarps : 0;
    const bool live = !SIDE || row < p.rows;

    Raw16<IN> x[NCH], r[RES ? NCH : 1];
    Raw16<WT> w[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int64_t k = (c * nwarps + warp) * kWarpVals + lane * kLaneVals;
        x[c].load(p.x + row * p.x_stride + k * E, live && k < K);
        if constexpr (RES)
            r[c].load(p.residual + row * p.residual_stride + k * E, live && k < K);
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int64_t k = (c * nwarps + warp) * kWarpVals + lane * kLaneVals;
        w[c].template load<true>(p.weight + k * ElemBytes<WT>::value, k < K);
    }
    F2 h[NCH][kLaneVals / 2], ss2 = f2(0.0f, 0.0f);
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int i = 0; i < kLaneVals / 2; ++i) {
            h[c][i] = x[c].pair(i);
            if constexpr (RES)
                h[c][i] = f2_add(h[c][i], r[c].pair(i));
            ss2 = f2_fma(h[c][i], h[c][i], ss2);
        }
    float ss, odd;
    f2_split(ss2, ss, odd);
    ss = warp_sum(ss + odd);
    if (lane == 0)
        part[part0 + warp] = ss;
    __syncthreads();
    ss = warp_sum(lane < nwarps ? part[part0 + lane] : 0.0f);
    const float rstd = __frsqrt_rn(ss / static_cast<float>(K) + p.eps);
    if (threadIdx.x == 0 && p.rstd && live)
        p.rstd[row] = rstd;
#pragma unroll
    for (int c = 0; c < NCH && live; ++c) {
        const int64_t k0 = (c * nwarps + warp) * kWarpVals;
        const int64_t k = k0 + lane * kLaneVals;
        const bool inside = k < K;
        float v[kLaneVals];
        if (p.h && inside) {
#pragma unroll
            for (int i = 0; i < kLaneVals / 2; ++i)
                f2_split(h[c][i], v[2 * i], v[2 * i + 1]);
            store16<IN>(p.h + (row * K + k) * E, v);
        }
#pragma unroll
        for (int i = 0; i < kLaneVals / 2; ++i)
            f2_split(f2_mul(f2_mul(h[c][i], f2(rstd, rstd)), w[c].pair(i)), v[2 * i], v[2 * i + 1]);
        if (p.y && inside)
            store16<IN>(p.y + (row * K + k) * E, v);
        if (FMT != kNoFmt) {
            const auto e = mx_encode<FMT == kNoFmt ? kMxfp8 : FMT>(v);
            if (inside)
                store_codes(p.mx.codes + row * (FMT == kMxfp8 ? K : K >> 1), k, e);
            store_scales(p.mx.scales, p.mx.mode, row, k0, K, lane, e.scode);
        }
    }
    if (FMT != kNoFmt && p.mx.mode == kScaleTiled)
        pad_tiled_scales(p.mx.scales, p.rows, K, row * blockDim.x + threadIdx.x,
                         static_cast<int64_t>(gridDim.x) * (SIDE ? blockDim.y : 1) * blockDim.x);
}

// ----------------------------------------------------------------- backward --
// Blocks stride over the rows; a thread sums its columns' share of dw and leaves it
// in partial[block].  Rows of more than 8192 values: two passes over the row, the
// second from L2, with dw in shared memory ([run][pair][thread], so that a warp's
// accesses are consecutive).
// dx of a pair of values; unit is h * rstd, coef -mean(p * unit) of the row
__device__ __forceinline__ F2 norm_dx(F2 dy, F2 unit, F2 dh, F2 w, F2 coef, F2 rstd)
{
    return f2_fma(f2_fma(unit, coef, f2_mul(dy, w)), rstd, dh);
}

constexpr int kWideThreads = 512;
constexpr int kWideVals = kWideThreads * kLaneVals;

template <int IN, int WT>
__global__ void __launch_bounds__(kWideThreads) rmsnorm_backward_wide_kernel(const NormBackParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    extern __shared__ __align__(16) F2 wide_dw[];
    __shared__ float part[2][32];
    griddep_launch_dependents();
    griddep_wait();
    const int64_t K = p.K, k0 = threadIdx.x * kLaneVals;
    F2 *const dw = wide_dw + threadIdx.x;
    int n = 0;
    for (int64_t k = k0; k < K; k += kWideVals, n += kLaneVals / 2)
#pragma unroll
        for (int i = 0; i < kLaneVals / 2; ++i)
            dw[(n + i) * kWideThreads] = f2(0.0f, 0.0f);
    int flip = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= 1) {
        const char *dy_row = p.dy + row * p.dy_stride, *h_row = p.h + row * p.h_stride;
        const float rstd = p.rstd[row];
        float dot = 0.0f;
#pragma unroll 2
        for (int64_t k = k0; k < K; k += kWideVals) {
            Raw16<IN> dy, h;
            Raw16<WT> w;
            dy.load(dy_row + k * E, true);
            h.load(h_row + k * E, true);
            w.template load<true>(p.weight + k * ElemBytes<WT>::value, true);
#pragma unroll
            for (int i = 0; i < kLaneVals; ++i)
                dot = fmaf(dy.at(i) * w.at(i), h.at(i), dot);
        }
        dot = block_sum(dot, part[flip]);
        const float coef = rstd * (dot / static_cast<float>(K));
        n = 0;
        for (int64_t k = k0; k < K; k += kWideVals, n += kLaneVals / 2) {
            Raw16<IN> dy, h, dh;
            Raw16<WT> w;
            dy.load(dy_row + k * E, true);
            h.load(h_row + k * E, true);
            dh.load(p.dh + row * p.dh_stride + k * E, p.dh != nullptr);
            w.template load<true>(p.weight + k * ElemBytes<WT>::value, true);
            float dx[kLaneVals];
#pragma unroll
            for (int i = 0; i < kLaneVals; i += 2) {
                F2 &sum = dw[(n + i / 2) * kWideThreads];
                const F2 g = dy.pair(i / 2), unit = f2_mul(h.pair(i / 2), f2(rstd, rstd));
                sum = f2_fma(g, unit, sum);
                f2_split(norm_dx(g, unit, dh.pair(i / 2), w.pair(i / 2), f2(-coef, -coef), f2(rstd, rstd)), dx[i],
                         dx[i + 1]);
            }
            store16<IN>(p.dx + (row * K + k) * E, dx);
        }
    }
    n = 0;
    for (int64_t k = k0; k < K; k += kWideVals, n += kLaneVals / 2) {
        float v[kLaneVals];
#pragma unroll
        for (int i = 0; i < kLaneVals; i += 2)
            f2_split(dw[(n + i / 2) * kWideThreads], v[i], v[i + 1]);
        store16<kF32>(reinterpret_cast<char *>(p.partial + blockIdx.x * K + k), v);
    }
}

// Rows of at most 8192 values (16 a thread), as a pipeline.  Each
// thread copies its own values of dy, h and dh of the coming rows to its own places
// in a ring in shared memory (cp.async) and reads them back itself, so the ring needs
// no barrier.  Between two barriers a block forms the dot product's partial sums of
// one row and finishes the row before it, whose sums the last barrier made visible:
// the reduction's latency is covered by work instead of being waited out.
// SIDE: blockDim.y rows beside each other, whose weight sums are joined at the end.
__device__ __forceinline__ void cp_async16(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// A thread's values come in 16-byte pieces `threads` pieces apart, so that a warp's
// copies are 512 consecutive bytes (two 16-byte halves of a 32-byte run per thread
// would fetch every sector twice).  The kernels for few and for many rows share this
// layout and these sums, so a row's dx does not depend on how many rows there are.
template <int IN>
struct Pieces {
    static constexpr int kPer = 16 / ElemBytes<IN>::value;  // values of a piece
    static constexpr int kCount = kLaneVals / kPer;         // pieces of a thread
    static constexpr int kPairs = kPer / 2;                 // FP32 pairs of a piece

    static __device__ __forceinline__ F2 pair(const uint4 &v, int n)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (IN == kBf16)
            return f2_bf16(w[n]);
        else
            return f2(__uint_as_float(w[2 * n]), __uint_as_float(w[2 * n + 1]));
    }

    // The weight at values k .. of this thread's piece.
    template <int WT>
    static __device__ __forceinline__ void load_weight(F2 (&w)[kPairs], const char *weight, uint32_t k, bool inside)
    {
#pragma unroll
        for (int n = 0; n < kPairs; ++n) {
            w[n] = f2(0.0f, 0.0f);
            if (inside) {
                if constexpr (WT == kBf16) {
                    w[n] = f2_bf16(reinterpret_cast<const uint32_t *>(weight)[k / 2 + n]);
                } else {
                    const float2 v = reinterpret_cast<const float2 *>(weight)[k / 2 + n];
                    w[n] = f2(v.x, v.y);
                }
            }
        }
    }

    // dot += dy * w * h of one piece
    static __device__ __forceinline__ F2 dot(F2 sum, const uint4 &dy, const uint4 &h, const F2 (&w)[kPairs])
    {
#pragma unroll
        for (int n = 0; n < kPairs; ++n)
            sum = f2_fma(f2_mul(pair(dy, n), w[n]), pair(h, n), sum);
        return sum;
    }

    static __device__ __forceinline__ uint4 pack(const F2 (&v)[kPairs])
    {
        float d[kPer];
#pragma unroll
        for (int n = 0; n < kPairs; ++n)
            f2_split(v[n], d[2 * n], d[2 * n + 1]);
        if constexpr (IN == kBf16)
            return make_uint4(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]), pack_bf16(d[4], d[5]),
                              pack_bf16(d[6], d[7]));
        else
            return make_uint4(__float_as_uint(d[0]), __float_as_uint(d[1]), __float_as_uint(d[2]),
                              __float_as_uint(d[3]));
    }
};

// A warp's share of a row's dot product into its entry; entries of warps that there
// are not hold zero.
__device__ __forceinline__ void leave_dot(F2 dot, float *part)
{
    float lo, hi;
    f2_split(dot, lo, hi);
    lo = warp_sum(lo + hi);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = lo;
}

// -mean(p * h * rstd) of a row
__device__ __forceinline__ float row_coef(const float *part, float rstd, float inv_k)
{
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kMaxThreads / 128; ++i) {
        const float4 v = reinterpret_cast<const float4 *>(part)[i];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    return -(rstd * (((s.x + s.y) + (s.z + s.w)) * inv_k));
}

template <int IN, int WT, int DEPTH, bool SIDE>
__global__ void __launch_bounds__(SIDE ? kSideThreads : kMaxThreads, SIDE ? 4 : 0)
    rmsnorm_backward_ring_kernel(const NormBackParams p)
{
    using P = Pieces<IN>;
    constexpr int E = ElemBytes<IN>::value, kPer = P::kPer, kPieces = P::kCount, kPairs = P::kPairs;
    constexpr int kSides = SIDE ? kSideThreads / 32 : 1;
    extern __shared__ __align__(16) uint4 ring[];  // [side][DEPTH][dy, h, dh][piece][thread]
    __shared__ __align__(16) float parts[kSides][2][kMaxThreads / 32];
    __shared__ float rstds[kSides][2];  // by thread 0, a row ahead; each iteration's barrier shows it to the others
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t threads = blockDim.x, tid = threadIdx.x, side = SIDE ? threadIdx.y : 0;
    const uint32_t sides = SIDE ? blockDim.y : 1;
    float(&part)[2][kMaxThreads / 32] = parts[side];
    float(&row_rstd)[2] = rstds[side];
    const int64_t K = p.K, step = static_cast<int64_t>(gridDim.x) * sides;
    const int64_t block_row = static_cast<int64_t>(blockIdx.x) * sides;
    const bool with_dh = p.dh != nullptr;
    const uint32_t plane = threads * 16;                                   // bytes of one piece of all threads
    const uint32_t stage_bytes = (with_dh ? 3 : 2) * kPieces * plane;
    const uint32_t ring0 = smem_addr(ring) + side * DEPTH * stage_bytes + tid * 16;
    const uint32_t ring_end = ring0 + DEPTH * stage_bytes;
    bool inside[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
        inside[i] = (i * threads + tid) * kPer < K;

    // the row that is fetched next, and where to
    int64_t ahead_row = block_row + side;
    const char *src_dy = p.dy + ahead_row * p.dy_stride + tid * 16, *src_h = p.h + ahead_row * p.h_stride + tid * 16,
               *src_dh = p.dh + ahead_row * p.dh_stride + tid * 16;
    uint32_t to = ring0;
    auto fetch = [&]() {
        if (ahead_row < p.rows) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                if (inside[i]) {
                    cp_async16(to + i * plane, src_dy + i * plane);
                    cp_async16(to + (kPieces + i) * plane, src_h + i * plane);
                    if (with_dh)
                        cp_async16(to + (2 * kPieces + i) * plane, src_dh + i * plane);
                }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ahead_row += step;
        src_dy += step * p.dy_stride;
        src_h += step * p.h_stride;
        src_dh += step * p.dh_stride;
        to += stage_bytes;
        to = to == ring_end ? ring0 : to;
    };
    if (tid < 2 * (kMaxThreads / 32))
        part[tid / (kMaxThreads / 32)][tid % (kMaxThreads / 32)] = 0.0f;  // for warps that there are not
    auto take = [&](uint32_t at, int i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (inside[i])
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(at)
                         : "memory");
        return v;
    };
#pragma unroll
    for (int d = 0; d < DEPTH - 1; ++d)
        fetch();
    F2 w[kPieces][kPairs], dw[kPieces][kPairs];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        P::template load_weight<WT>(w[i], p.weight, (i * threads + tid) * kPer, inside[i]);
#pragma unroll
        for (int n = 0; n < kPairs; ++n)
            dw[i][n] = f2(0.0f, 0.0f);
    }
    uint4 next_dy[kPieces], next_h[kPieces];
    // partial sums of p * h of a row that has landed; its dy and h stay in registers for its turn
    auto dot_row = [&](uint32_t from, int buf) {
        F2 dot = f2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            next_dy[i] = take(from + i * plane, i);
            next_h[i] = take(from + (kPieces + i) * plane, i);
            dot = P::dot(dot, next_dy[i], next_h[i], w[i]);
        }
        leave_dot(dot, part[buf]);
    };
    int64_t row = block_row + side;
    char *dx = p.dx + row * K * E + tid * 16;
    float next_rstd = 0.0f;
    if (tid == 0 && row < p.rows) {
        row_rstd[0] = p.rstd[row];
        next_rstd = row + step < p.rows ? p.rstd[row + step] : 0.0f;
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory");
    __syncthreads();
    dot_row(ring0, 0);
    __syncthreads();
    const float inv_k = 1.0f / static_cast<float>(K);
    uint32_t stage = ring0;
    int buf = 0;
    for (; row - side < p.rows; row += step, buf ^= 1) {  // all sides of a block take part in its barriers
        uint32_t following = stage + stage_bytes;
        following = following == ring_end ? ring0 : following;
        fetch();  // into the stage that the last row left
        const float rstd = row_rstd[buf];
        if (tid == 0) {
            row_rstd[buf ^ 1] = next_rstd;
            next_rstd = row + 2 * step < p.rows ? p.rstd[row + 2 * step] : 0.0f;
        }
        const float coef = row_coef(part[buf], rstd, inv_k);
        uint4 dy[kPieces], h[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            dy[i] = next_dy[i];
            h[i] = next_h[i];
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory");
        if (row + step < p.rows)
            dot_row(following, buf ^ 1);
        const F2 coef2 = f2(coef, coef), rstd2 = f2(rstd, rstd);
        const bool live = !SIDE || row < p.rows;
#pragma unroll
        for (int i = 0; i < kPieces && live; ++i) {
            uint4 dh = make_uint4(0, 0, 0, 0);
            if (with_dh)
                dh = take(stage + (2 * kPieces + i) * plane, i);
            F2 o[kPairs];
#pragma unroll
            for (int n = 0; n < kPairs; ++n) {
                const F2 g = P::pair(dy[i], n), unit = f2_mul(P::pair(h[i], n), rstd2);
                o[n] = norm_dx(g, unit, P::pair(dh, n), w[i][n], coef2, rstd2);
                dw[i][n] = f2_fma(g, unit, dw[i][n]);
            }
            if (inside[i])
                *reinterpret_cast<uint4 *>(dx + i * plane) = P::pack(o);
        }
        dx += step * K * E;
        stage = following;
        __syncthreads();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if constexpr (SIDE) {  // the sides' sums in order, through the ring that nothing uses any more
        __syncthreads();
        F2 *const sums = reinterpret_cast<F2 *>(ring) + tid;
        if (side > 0)
#pragma unroll
            for (int i = 0; i < kPieces * kPairs; ++i)
                sums[((side - 1) * kPieces * kPairs + i) * threads] = dw[i / kPairs][i % kPairs];
        __syncthreads();
        if (side > 0)
            return;
        for (uint32_t other = 0; other + 1 < sides; ++other)
#pragma unroll
            for (int i = 0; i < kPieces * kPairs; ++i)
                dw[i / kPairs][i % kPairs] =
                    f2_add(dw[i / kPairs][i % kPairs], sums[(other * kPieces * kPairs + i) * threads]);
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
        if (inside[i]) {
            float *out = p.partial + blockIdx.x * K + (i * threads + tid) * kPer;
#pragma unroll
            for (int n = 0; n < kPairs; n += 2) {
                float4 o;
                f2_split(dw[i][n], o.x, o.y);
                f2_split(dw[i][n + 1], o.z, o.w);
                *reinterpret_cast<float4 *>(out + 2 * n) = o;
            }
        }
}

// dw[k] = sum of partial[b][k] over the blocks, in block order within each of 32
// slices and then over the slices: the same sum every run.
constexpr int kSlices = 32;  // as many as columns of a block: warp s finishes column s

__global__ void __launch_bounds__(32 * kSlices)
    rmsnorm_dweight_kernel(const float *partial, int blocks, int64_t K, float *dw)
{
    __shared__ float part[kSlices][33];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t k0 = static_cast<int64_t>(blockIdx.x) * 32, k = k0 + lane;
    float v = 0.0f;
#pragma unroll 10
    for (int b = slice; b < blocks; b += kSlices)
        v += partial[b * K + k];
    part[slice][lane] = v;
    __syncthreads();
    v = warp_sum(part[lane][slice]);  // warp `slice` adds column `slice` over the slices
    if (lane == 0)
        dw[k0 + slice] = v;
}

// Few rows: dw needs no dx, so one launch does both.  The first blocks sum the
// columns' products over all rows (two neighbouring columns a lane in BF16, one in
// FP32, the rows dealt to the warps), the others take a row each; dy and h are read
// twice, the second time from L2, and there is neither a second launch nor partial
// sums to wait for (all with dh): 64 x 4096 BF16 2.6 us against 5.6 with the ring, 301 x
// 4096 FP32 6.5 against 9.7, 1024 BF16 rows of 1024 to 8192 values 6.9-15.0 against
// 7.4-18.4; from 2048 rows on the columns' blocks are too long (2048 x 1024: 15.2 against
// 10.1).  Two blocks an SM (64 registers): with one, 301 x 5120 FP32 takes 11.8 us instead
// of 7.6.  What binds it is the number of blocks that fit at once, 304 of those 461: all
// have 512 threads, of which a row of 5120 values uses 320.
constexpr int64_t kFewRows = 1024;

template <int IN, int WT>
__global__ void __launch_bounds__(kMaxThreads, 2) rmsnorm_backward_few_kernel(const NormBackParams p, int column_blocks)
{
    using P = Pieces<IN>;
    constexpr int E = ElemBytes<IN>::value;
    constexpr int kCols = IN == kBf16 ? 64 : 32;
    __shared__ __align__(16) float part[kMaxThreads / 32];
    __shared__ float2 sums[kMaxThreads / 32][32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int64_t K = p.K;
    if (static_cast<int>(blockIdx.x) < column_blocks) {
        const int64_t k = static_cast<int64_t>(blockIdx.x) * kCols + lane * (kCols / 32);
        const char *dy = p.dy + k * E, *h = p.h + k * E;
        float2 sum = make_float2(0.0f, 0.0f);
        if (k < K)
#pragma unroll 8
            for (int64_t row = warp; row < p.rows; row += nwarps) {
                const float rstd = p.rstd[row];
                if constexpr (IN == kBf16) {
                    const uint32_t g = *reinterpret_cast<const uint32_t *>(dy + row * p.dy_stride);
                    const uint32_t v = *reinterpret_cast<const uint32_t *>(h + row * p.h_stride);
                    sum.x = fmaf(__uint_as_float(g << 16), __uint_as_float(v << 16) * rstd, sum.x);
                    sum.y = fmaf(__uint_as_float(g & 0xFFFF0000u), __uint_as_float(v & 0xFFFF0000u) * rstd, sum.y);
                } else {
                    sum.x = fmaf(*reinterpret_cast<const float *>(dy + row * p.dy_stride),
                                 *reinterpret_cast<const float *>(h + row * p.h_stride) * rstd, sum.x);
                }
            }
        sums[warp][lane] = sum;
        __syncthreads();
        if (warp == 0 && k < K) {
            for (int w = 1; w < nwarps; ++w) {
                sum.x += sums[w][lane].x;
                sum.y += sums[w][lane].y;
            }
            if constexpr (IN == kBf16)
                *reinterpret_cast<float2 *>(p.dweight + k) = sum;
            else
                p.dweight[k] = sum.x;
        }
        return;
    }
    const int64_t row = blockIdx.x - column_blocks;
    const uint32_t threads = (static_cast<uint32_t>(K) + kWarpVals - 1) / kWarpVals * 32, tid = threadIdx.x;
    uint4 dy[P::kCount], h[P::kCount], dh[P::kCount];
    F2 w[P::kCount][P::kPairs], dot = f2(0.0f, 0.0f);
    bool inside[P::kCount];
#pragma unroll
    for (int i = 0; i < P::kCount; ++i) {
        const uint32_t k = (i * threads + tid) * P::kPer;
        inside[i] = tid < threads && k < K;
        dy[i] = h[i] = dh[i] = make_uint4(0, 0, 0, 0);
        if (inside[i]) {
            dy[i] = *reinterpret_cast<const uint4 *>(p.dy + row * p.dy_stride + static_cast<int64_t>(k) * E);
            h[i] = *reinterpret_cast<const uint4 *>(p.h + row * p.h_stride + static_cast<int64_t>(k) * E);
        }
        P::template load_weight<WT>(w[i], p.weight, k, inside[i]);
    }
    // dh is needed last: in FP32 its registers would be one block less on an SM, so it is loaded after the sum
    auto load_dh = [&]() {
        if (p.dh)
#pragma unroll
            for (int i = 0; i < P::kCount; ++i)
                if (inside[i])
                    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(dh[i].x), "=r"(dh[i].y), "=r"(dh[i].z), "=r"(dh[i].w)
                                 : "l"(p.dh + row * p.dh_stride + ((i * threads + tid) * P::kPer) * E)
                                 : "memory");
    };
    if (IN == kBf16)
        load_dh();
    const float rstd = p.rstd[row];
#pragma unroll
    for (int i = 0; i < P::kCount; ++i)
        dot = P::dot(dot, dy[i], h[i], w[i]);
    leave_dot(dot, part);
    if (IN != kBf16)
        load_dh();
    __syncthreads();
    const float coef = row_coef(part, rstd, 1.0f / static_cast<float>(K));
#pragma unroll
    for (int i = 0; i < P::kCount; ++i) {
        F2 o[P::kPairs];
#pragma unroll
        for (int n = 0; n < P::kPairs; ++n)
            o[n] = norm_dx(P::pair(dy[i], n), f2_mul(P::pair(h[i], n), f2(rstd, rstd)), P::pair(dh[i], n), w[i][n],
                           f2(coef, coef), f2(rstd, rstd));
        if (inside[i])
            *reinterpret_cast<uint4 *>(p.dx + (row * K + (i * threads + tid) * P::kPer) * E) = P::pack(o);
    }
}

// Runs of 16 values a thread takes of a row of K values, at least `least`, with at
// most kMaxThreads threads.
struct Shape {
    int nch, threads;
};

Shape pick_shape(int64_t K, int least = 1)
{
    Shape s;
    s.nch = K <= 8192 && least == 1 ? 1 : K <= 16384 ? 2 : 4;
    const int64_t warps = (K + s.nch * kWarpVals - 1) / (s.nch * kWarpVals);
    s.threads = static_cast<int>(warps) * 32;
    return s;
}

// Backward: rows of up to 8192 values take the ring, with 512 threads' worth of
// blocks on an SM (four at most); wider ones as many blocks as their sums in shared
// memory allow, two at most (each leaves a row of partial sums).
constexpr int64_t kRingMaxK = 8192;  // kMaxThreads threads' values
bool few_rows(int64_t rows, int64_t K) { return K <= kRingMaxK && rows <= kFewRows; }
int blocks_per_sm(int64_t K)
{
    if (K > kRingMaxK)
        return K <= 2 * kWideVals ? 2 : 1;
    const int n = 512 / pick_shape(K).threads;
    return n > 4 ? 4 : n;
}

// BF16 without a residual brings half the bytes to hide a row's reduction behind, and
// instructions bind as well: a thread takes 32 values to spread the fixed ones over
// (16384 x 8192 to MXFP8: 73 us, 87 with 16).  Elsewhere 16 are as good or better (with
// a residual 135 us either way).
template <int IN, bool RES>
constexpr int fewest_runs()
{
    return IN == kBf16 && !RES ? 2 : 1;
}

template <int IN, int WT, int FMT, int NCH, bool RES>
cudaError_t launch_rows(const NormParams &p, int threads, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    constexpr bool kNarrow = NCH == fewest_runs<IN, RES>();
    const int side = kNarrow && p.K <= kSideK && p.rows >= kSideRows ? kSideThreads / threads : 1;
    cudaLaunchConfig_t cfg = row_launch(static_cast<unsigned>((p.rows + side - 1) / side), threads, 0, s, attr);
    if constexpr (kNarrow)
        if (side > 1) {
            cfg.blockDim.y = side;
            return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<IN, WT, FMT, NCH, RES, true>, p);
        }
    return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<IN, WT, FMT, NCH, RES, false>, p);
}

template <int IN, int WT, int FMT, bool RES>
cudaError_t launch_forward(const NormParams &p, cudaStream_t s)
{
    constexpr int kLeast = fewest_runs<IN, RES>();
    const Shape sh = pick_shape(p.K, kLeast);
    if constexpr (kLeast == 1)
        if (sh.nch == 1)
            return launch_rows<IN, WT, FMT, 1, RES>(p, sh.threads, s);
    return sh.nch == 2 ? launch_rows<IN, WT, FMT, 2, RES>(p, sh.threads, s)
                       : launch_rows<IN, WT, FMT, 4, RES>(p, sh.threads, s);
}

template <int IN, int WT, int FMT>
cudaError_t launch_forward_res(const NormParams &p, cudaStream_t s)
{
    return p.residual ? launch_forward<IN, WT, FMT, true>(p, s) : launch_forward<IN, WT, FMT, false>(p, s);
}

template <int IN, int WT>
cudaError_t launch_forward_fmt(const NormParams &p, cudaStream_t s)
{
    return p.mx.fmt == kMxfp8   ? launch_forward_res<IN, WT, kMxfp8>(p, s)
           : p.mx.fmt == kMxfp4 ? launch_forward_res<IN, WT, kMxfp4>(p, s)
                                : launch_forward_res<IN, WT, kNoFmt>(p, s);
}

constexpr int kRingBytes = 220 * 1024;  // shared memory of an SM's rings

template <int IN, int WT, int DEPTH>
cudaError_t launch_ring(const NormBackParams &p, int threads, int sides, int64_t blocks, size_t smem, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = row_launch(static_cast<unsigned>(blocks), threads, smem, s, attr);
    cfg.blockDim.y = sides;
    if constexpr (IN == kBf16 && DEPTH == 4)
        if (sides > 1)
            return cudaLaunchKernelEx(&cfg, rmsnorm_backward_ring_kernel<IN, WT, DEPTH, true>, p);
    return cudaLaunchKernelEx(&cfg, rmsnorm_backward_ring_kernel<IN, WT, DEPTH, false>, p);
}

// Narrow rows (up to 1024 values) in BF16 share a block, two or four at a time: 16384 x
// 992 29 us with dh, 40 with a row a block, 25 and 36 without.  In FP32 the registers for
// that spill (8192 x 992: 36 us against 29).  Blocks of 128 threads that read dh run best
// three to an SM (16384 x 2048: 52 us, 59 with four), those that do not with four (41 us, 45).
template <int IN, int WT>
cudaError_t launch_backward(const NormBackParams &p, int num_sms, cudaStream_t s)
{
    const Shape sh = pick_shape(p.K);
    const int sides = IN == kBf16 && p.K <= kSideK ? kSideThreads / sh.threads : 1;
    int64_t blocks = norm_back_blocks(p.rows, p.K);
    int per_sm = blocks_per_sm(p.K);
    if (p.dh && per_sm == 4 && sh.threads * sides == 128)
        per_sm = 3;
    blocks = blocks < static_cast<int64_t>(num_sms) * per_sm ? blocks : static_cast<int64_t>(num_sms) * per_sm;
    cudaError_t e;
    cudaLaunchAttribute attr[1];
    if (few_rows(p.rows, p.K)) {
        const int columns = static_cast<int>((p.K + (IN == kBf16 ? 63 : 31)) / (IN == kBf16 ? 64 : 32));
        const cudaLaunchConfig_t cfg = row_launch(static_cast<unsigned>(columns + p.rows), kMaxThreads, 0, s, attr);
        return cudaLaunchKernelEx(&cfg, rmsnorm_backward_few_kernel<IN, WT>, p, columns);
    }
    if (p.K <= kRingMaxK) {
        const int64_t row = static_cast<int64_t>(p.dh ? 3 : 2) * sides * sh.threads * kLaneVals * ElemBytes<IN>::value;
        // an SM's blocks have at most 512 threads: their stages take at most 48 KB in BF16, 96 in FP32
        if constexpr (IN == kBf16) {
            e = launch_ring<IN, WT, 4>(p, sh.threads, sides, blocks, 4 * row, s);
        } else {
            const int64_t depth = kRingBytes / per_sm / row;
            e = depth >= 4   ? launch_ring<IN, WT, 4>(p, sh.threads, sides, blocks, 4 * row, s)
                : depth == 3 ? launch_ring<IN, WT, 3>(p, sh.threads, sides, blocks, 3 * row, s)
                             : launch_ring<IN, WT, 2>(p, sh.threads, sides, blocks, 2 * row, s);
        }
    } else {
        const size_t smem = (p.K + kWideVals - 1) / kWideVals * kWideVals * sizeof(float);
        const cudaLaunchConfig_t cfg = row_launch(static_cast<unsigned>(blocks), kWideThreads, smem, s, attr);
        e = cudaLaunchKernelEx(&cfg, rmsnorm_backward_wide_kernel<IN, WT>, p);
    }
    if (e != cudaSuccess)
        return e;
    const cudaLaunchConfig_t cfg = row_launch(static_cast<unsigned>(p.K / 32), 32 * kSlices, 0, s, attr);
    return cudaLaunchKernelEx(&cfg, rmsnorm_dweight_kernel, static_cast<const float *>(p.partial),
                              static_cast<int>(blocks), p.K, p.dweight);
}

template <int IN, int WT>
cudaError_t prepare_backward()
{
    constexpr auto kAttr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(rmsnorm_backward_ring_kernel<IN, WT, 4, false>, kAttr, kRingBytes);
    if constexpr (IN == kBf16) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(rmsnorm_backward_ring_kernel<IN, WT, 4, true>, kAttr, kRingBytes);
    } else {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(rmsnorm_backward_ring_kernel<IN, WT, 3, false>, kAttr, kRingBytes);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(rmsnorm_backward_ring_kernel<IN, WT, 2, false>, kAttr, kRingBytes);
    }
    return e == cudaSuccess ? cudaFuncSetAttribute(rmsnorm_backward_wide_kernel<IN, WT>, kAttr,
                                                   static_cast<int>(kNormMaxK * sizeof(float)))
                            : e;
}

}  // namespace

cudaError_t prepare_norm()
{
    cudaError_t e = prepare_backward<kBf16, kBf16>();
    if (e == cudaSuccess)
        e = prepare_backward<kBf16, kF32>();
    if (e == cudaSuccess)
        e = prepare_backward<kF32, kBf16>();
    return e == cudaSuccess ? prepare_backward<kF32, kF32>() : e;
}

int64_t norm_back_blocks(int64_t rows, int64_t K)
{
    if (few_rows(rows, K))
        return 0;
    const int64_t most = static_cast<int64_t>(kNormBackSms) * blocks_per_sm(K);
    return rows < most ? rows : most;
}

cudaError_t launch_rmsnorm(const NormParams &p, int in_dtype, int weight_dtype, cudaStream_t s)
{
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
