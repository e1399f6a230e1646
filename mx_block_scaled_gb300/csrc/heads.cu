// heads.cu -- RMS norm of query and key heads with the rotation of their
// positions, and its gradient.
//
//   n = x * rstd, rstd = 1/sqrt(mean(x^2) + eps) over a head;  y = R(position) (n * w)
//   g = R(-position) dy;  dx = rstd * (g * w - n * mean(g * w * n));  dw = sum over heads of g * n
//
// R turns the first `rotary` values of a head in pairs (a, b) -> (a cos - b sin, b cos + a sin),
// which are i and i + rotary/2, or 2i and 2i + 1.  A lane holds sixteen values of a
// head in which every pair is whole (two runs of eight), and their eight angles are
// the same eight consecutive ones in both orders: nothing but the two sums crosses
// lanes.  A head takes a team of 4 to 32 lanes, a warp walks over the heads of a
// token and keeps the token's angles in registers.
#include "mx_block.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// Eight consecutive values as loaded: 16 bytes in BF16, 32 in FP32.
template <int DT>
struct Raw8 {
    static constexpr int kWords = DT == kBf16 ? 4 : 8;
    uint32_t r[kWords];

    __device__ __forceinline__ void load(const char *p, bool inside)
    {
        if (!inside) {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                r[i] = 0;
        } else if constexpr (DT == kBf16) {
            asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                         : "l"(p)
                         : "memory");
        } else {
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                           "=r"(r[7])
                         : "l"(p)
                         : "memory");
        }
    }
    __device__ __forceinline__ float at(int i) const
    {
        if constexpr (DT == kBf16)
            return __uint_as_float((i & 1) ? (r[i >> 1] & 0xFFFF0000u) : (r[i >> 1] << 16));
        else
            return __uint_as_float(r[i]);
    }
};

template <int DT>
__device__ __forceinline__ void store8(char *p, const float *v)
{
    if constexpr (DT == kBf16) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = __float_as_uint(v[i]);
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    }
}

// A lane's place in a head: first values of its two runs of eight, and its angles.
struct Place {
    int a, b;
    int angle;     // first of its eight angles
    bool inside;   // the lane holds values of the head
    bool turned;   // and they are rotated

    __device__ __forceinline__ Place(int lane, int D, int rotary, bool interleaved)
    {
        const int halves = rotary / 16;  // lanes with rotated values
        inside = lane < D / 16;
        turned = lane < halves;
        angle = 8 * lane;
        if (turned && !interleaved) {
            a = 8 * lane;
            b = rotary / 2 + 8 * lane;
        } else {
            a = 16 * lane;
            b = 16 * lane + 8;
        }
    }
};

// Sum over the lanes of a team (a power of two of them).
__device__ __forceinline__ float team_sum(float v, int team)
{
    for (int o = team >> 1; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// v = runs a (0..7) and b (8..15); turned by the angles' cosines and sines (inverse: by minus the angles).
template <bool INTERLEAVED>
__device__ __forceinline__ void turn(float (&v)[16], const float (&cs)[8], const float (&sn)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int p = INTERLEAVED ? 2 * i : i, q = INTERLEAVED ? 2 * i + 1 : i + 8;
        const float x = v[p], y = v[q];
        v[p] = x * cs[i] - y * sn[i];
        v[q] = y * cs[i] + x * sn[i];
    }
}

// The angles of a token: false where its position is outside the table.
__device__ __forceinline__ bool load_angles(const HeadsCommon &p, const Place &at, int64_t token, float (&cs)[8],
                                            float (&sn)[8], bool inverse)
{
    bool real = true;
    int64_t position = 0;
    if (p.rope) {
        position = p.positions64 ? static_cast<const int64_t *>(p.positions)[token]
                                 : static_cast<const int32_t *>(p.positions)[token];
        real = position >= 0 && position < p.rope_rows;
    }
    const bool take = p.rope && real && at.turned;
    const char *row = reinterpret_cast<const char *>(p.rope + position * p.rotary + at.angle);
    Raw8<kF32> c, s;
    c.load(row, take);
    s.load(row + p.rotary / 2 * 4, take);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cs[i] = take ? c.at(i) : 1.0f;
        sn[i] = take ? (inverse ? -s.at(i) : s.at(i)) : 0.0f;
    }
    return real;
}

// Which weight a head takes (one past the last head: any that there is).
__device__ __forceinline__ bool is_query(const HeadsCommon &p, int h)
{
    return h < p.q_heads || p.q_heads == p.heads;
}

// Type of the weights of heads that are only rotated.
constexpr int kNoWeight = 0;

template <int WT>
__device__ __forceinline__ void load_weight(float (&w)[16], const HeadsCommon &p, const Place &at, bool query)
{
    if constexpr (WT != kNoWeight) {
        constexpr int E = ElemBytes<WT>::value;
        const char *from = query ? p.q_weight : p.k_weight;
        Raw8<WT> a, b;
        a.load(from + at.a * E, at.inside);
        b.load(from + at.b * E, at.inside);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = a.at(i);
            w[8 + i] = b.at(i);
        }
    }
}

// ------------------------------------------------------------------ forward --
// (and, without weights and by minus the angles, the gradient of the rotation alone)
// A warp takes `steps` groups of neighbouring heads of a token; the next group is
// loaded before the current one is finished.
template <int IN, int WT, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) heads_kernel(const HeadsParams p, int team, int steps, uint32_t per_token)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5), token = unit / per_token;
    if (token >= p.tokens)
        return;
    const int lane = threadIdx.x & 31, member = lane & (team - 1), side = 32 / team;
    const Place at(member, p.D, p.rotary, INTERLEAVED);
    const int first = static_cast<int>(unit - token * per_token) * steps * side + lane / team;
    const int last = first + steps * side;  // heads first, first + side, ..
    const char *x = p.x + token * p.x_token;
    Raw8<IN> a, b;
    a.load(x + first * p.x_head + at.a * E, at.inside && first < p.heads);
    b.load(x + first * p.x_head + at.b * E, at.inside && first < p.heads);
    float cs[8], sn[8], w[16];
    const bool real = load_angles(p, at, token, cs, sn, p.inverse);
    bool query = is_query(p, first);
    load_weight<WT>(w, p, at, query);
    const float inv_d = 1.0f / static_cast<float>(p.D);
    for (int h = first; h - lane / team < p.heads && h < last; h += side) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = a.at(i);
            v[8 + i] = b.at(i);
        }
        const int next = h + side;
        const bool more = at.inside && next < p.heads && next < last;
        a.load(x + next * p.x_head + at.a * E, more);
        b.load(x + next * p.x_head + at.b * E, more);
        const bool live = h < p.heads;
        if constexpr (WT != kNoWeight) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                ss = fmaf(v[i], v[i], ss);
            ss = team_sum(ss, team);
            const float rstd = __frsqrt_rn(ss * inv_d + p.eps);
            if (member == 0 && p.rstd && live)
                p.rstd[token * static_cast<int64_t>(p.heads) + h] = real ? rstd : 0.0f;
            if (query != is_query(p, h)) {
                query = false;
                load_weight<WT>(w, p, at, false);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = v[i] * rstd * w[i];
        }
        turn<INTERLEAVED>(v, cs, sn);
        if (!real)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = 0.0f;
        if (at.inside && live) {
            char *y = p.y + token * p.y_token + h * p.y_head;
            store8<IN>(y + at.a * E, v);
            store8<IN>(y + at.b * E, v + 8);
        }
    }
}

// ----------------------------------------------------------------- backward --
// Blocks stride over (token, group of heads) and keep the sums for both weights in
// registers; each leaves its sums in partial[block][query, key][D].
template <int IN, int WT, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 3) heads_backward_kernel(const HeadsBackParams p, int team)
{
    constexpr int E = ElemBytes<IN>::value;
    extern __shared__ float sums[];  // [kWarps][2][D]
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, member = lane & (team - 1), side = 32 / team;
    const Place at(member, p.D, p.rotary, INTERLEAVED);
    const float inv_d = 1.0f / static_cast<float>(p.D);
    float dq[16], dk[16], w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        dq[i] = dk[i] = 0.0f;
    bool query = is_query(p, 0);
    load_weight<WT>(w, p, at, is_query(p, 0));
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t token = static_cast<int64_t>(blockIdx.x) * kWarps + warp; token < p.tokens; token += step) {
        float cs[8], sn[8];
        const char *x = p.x + token * p.x_token, *dy = p.dy + token * p.dy_token;
        const int first = lane / team;
        Raw8<IN> xa, xb, ga, gb;
        float rstd;
        auto fetch = [&](int h) {
            const bool take = at.inside && h < p.heads;
            xa.load(x + h * p.x_head + at.a * E, take);
            xb.load(x + h * p.x_head + at.b * E, take);
            ga.load(dy + h * p.dy_head + at.a * E, take);
            gb.load(dy + h * p.dy_head + at.b * E, take);
            rstd = h < p.heads ? p.rstd[token * p.heads + h] : 0.0f;
        };
        fetch(first);
        const bool real = load_angles(p, at, token, cs, sn, true);
        for (int h = first; h - first < p.heads; h += side) {
            float n[16], g[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                n[i] = xa.at(i) * rstd;
                n[8 + i] = xb.at(i) * rstd;
                g[i] = ga.at(i);
                g[8 + i] = gb.at(i);
            }
            const float r = rstd;
            fetch(h + side);
            const bool q = is_query(p, h);
            if (q != query) {
                query = q;
                load_weight<WT>(w, p, at, q);
            }
            turn<INTERLEAVED>(g, cs, sn);
            if (!real)  // nothing of such a token counts, whatever its memory holds
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    n[i] = g[i] = 0.0f;
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                dot = fmaf(g[i] * w[i], n[i], dot);
            dot = team_sum(dot, team) * inv_d;
            if (q) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    dq[i] = fmaf(g[i], n[i], dq[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    dk[i] = fmaf(g[i], n[i], dk[i]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                g[i] = (g[i] * w[i] - n[i] * dot) * r;
            if (!real)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    g[i] = 0.0f;
            if (at.inside && h < p.heads) {
                char *dx = p.dx + token * p.dx_token + h * p.dx_head;
                store8<IN>(dx + at.a * E, g);
                store8<IN>(dx + at.b * E, g + 8);
            }
        }
    }
    // over the teams of the warp, then over the warps in order
    for (int o = team; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            dq[i] += __shfl_xor_sync(0xFFFFFFFFu, dq[i], o);
            dk[i] += __shfl_xor_sync(0xFFFFFFFFu, dk[i], o);
        }
    if (lane < team && at.inside) {
        float *mine = sums + warp * 2 * p.D;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            mine[at.a + i] = dq[i];
            mine[at.b + i] = dq[8 + i];
            mine[p.D + at.a + i] = dk[i];
            mine[p.D + at.b + i] = dk[8 + i];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            v += sums[w * 2 * p.D + i];
        p.partial[static_cast<int64_t>(blockIdx.x) * 2 * p.D + i] = v;
    }
}

// The blocks' sums in a fixed order: 32 slices of blocks a column, then the slices.
constexpr int kSlices = 32;

__global__ void __launch_bounds__(32 * kSlices)
    heads_dweight_kernel(const float *partial, int blocks, int D, float *dq, float *dk)
{
    __shared__ float part[kSlices][33];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int k0 = static_cast<int>(blockIdx.x) * 32;
    float v = 0.0f;
#pragma unroll 10
    for (int b = slice; b < blocks; b += kSlices)
        v += partial[static_cast<int64_t>(b) * 2 * D + k0 + lane];
    part[slice][lane] = v;
    __syncthreads();
    v = warp_sum(part[lane][slice]);  // warp `slice` adds column `slice` over the slices
    const int k = k0 + slice;
    if (lane == 0) {
        float *out = k < D ? dq : dk;
        if (out)
            out[k < D ? k : k - D] = v;
    }
}

int team_of(int D)
{
    int team = 1;
    while (team < D / 16)
        team *= 2;
    return team;
}

template <int IN, int WT>
cudaError_t launch_forward(const HeadsParams &p, bool interleaved, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const int team = team_of(p.D), side = 32 / team, groups = (p.heads + side - 1) / side;
    // all heads of a token to a warp where that leaves every multiprocessor sixteen warps; else fewer, down to one group
    int parts = 1;
    while (parts < groups && p.tokens * parts < 16ll * num_sms)
        ++parts;
    const int steps = (groups + parts - 1) / parts;
    const uint32_t per_token = static_cast<uint32_t>((groups + steps - 1) / steps);
    const int64_t warps = p.tokens * per_token;
    const cudaLaunchConfig_t cfg =
        row_launch(static_cast<unsigned>((warps + kWarps - 1) / kWarps), kThreads, 0, s, attr);
    return interleaved ? cudaLaunchKernelEx(&cfg, heads_kernel<IN, WT, true>, p, team, steps, per_token)
                       : cudaLaunchKernelEx(&cfg, heads_kernel<IN, WT, false>, p, team, steps, per_token);
}

template <int IN, int WT>
cudaError_t launch_backward(const HeadsBackParams &p, bool interleaved, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    int64_t blocks = heads_back_blocks(p.tokens);
    const int64_t most = static_cast<int64_t>(num_sms) * kHeadsBackPerSm;
    blocks = blocks < most ? blocks : most;
    cudaLaunchConfig_t cfg = row_launch(static_cast<unsigned>(blocks), kThreads,
                                        static_cast<size_t>(kWarps) * 2 * p.D * sizeof(float), s, attr);
    const int team = team_of(p.D);
    const cudaError_t e = interleaved ? cudaLaunchKernelEx(&cfg, heads_backward_kernel<IN, WT, true>, p, team)
                                      : cudaLaunchKernelEx(&cfg, heads_backward_kernel<IN, WT, false>, p, team);
    if (e != cudaSuccess)
        return e;
    cfg = row_launch(static_cast<unsigned>(p.D / 16), 32 * kSlices, 0, s, attr);
    return cudaLaunchKernelEx(&cfg, heads_dweight_kernel, static_cast<const float *>(p.partial),
                              static_cast<int>(blocks), p.D, p.dq_weight, p.dk_weight);
}

}  // namespace

int64_t heads_back_blocks(int64_t tokens)
{
    const int64_t blocks = (tokens + kWarps - 1) / kWarps, most = static_cast<int64_t>(kHeadsBackSms) * kHeadsBackPerSm;
    return blocks < most ? blocks : most;
}

cudaError_t launch_heads(const HeadsParams &p, int in_dtype, int weight_dtype, bool interleaved, int num_sms,
                         cudaStream_t s)
{
    if (in_dtype == kBf16)
        return weight_dtype == kNoWeight ? launch_forward<kBf16, kNoWeight>(p, interleaved, num_sms, s)
               : weight_dtype == kBf16   ? launch_forward<kBf16, kBf16>(p, interleaved, num_sms, s)
                                         : launch_forward<kBf16, kF32>(p, interleaved, num_sms, s);
    return weight_dtype == kNoWeight ? launch_forward<kF32, kNoWeight>(p, interleaved, num_sms, s)
           : weight_dtype == kBf16   ? launch_forward<kF32, kBf16>(p, interleaved, num_sms, s)
                                     : launch_forward<kF32, kF32>(p, interleaved, num_sms, s);
}

cudaError_t launch_heads_backward(const HeadsBackParams &p, int in_dtype, int weight_dtype, bool interleaved,
                                  int num_sms, cudaStream_t s)
{
    if (in_dtype == kBf16)
        return weight_dtype == kBf16 ? launch_backward<kBf16, kBf16>(p, interleaved, num_sms, s)
                                     : launch_backward<kBf16, kF32>(p, interleaved, num_sms, s);
    return weight_dtype == kBf16 ? launch_backward<kF32, kBf16>(p, interleaved, num_sms, s)
                                 : launch_backward<kF32, kF32>(p, interleaved, num_sms, s);
}

}  // namespace mxg
