// mx_block.cuh -- device helpers of the row operators (norm.cu, glu.cu, moe.cu):
// 32-byte row accesses and the MX encoding of values that a warp holds in
// registers.
//
// Layout every helper assumes: a warp owns 512 consecutive values of one row,
// lane l the sixteen from 16*l on, so the two lanes of an even/odd pair hold one
// 32-value scale block and eight lanes one 128-value K-tile.  Row lengths are
// multiples of 32: a pair of lanes is inside the row or outside it together.
// The encoding is mxgemm_quantize's recipe on FP32 values: scale exponent
// floor(log2 amax) - e_max (8 for E4M3, 2 for E2M1) not below -127, codes
// rounded to nearest even and saturated, a block with a NaN or an infinity as
// scale code 0xFF and zero codes.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace mxg {

constexpr int kLaneVals = 16;                // values a lane holds
constexpr int kWarpVals = 32 * kLaneVals;    // values of a warp's chunk

// Element types of plain operands and formats of encoded ones (as in mxgemm.h).
constexpr int kF32 = 1;
constexpr int kBf16 = 2;
constexpr int kNoFmt = 0;
constexpr int kMxfp8 = 1;
constexpr int kMxfp4 = 2;
constexpr int kRowsBf16 = 3;

template <int DT>
struct ElemBytes {
    static constexpr int value = DT == kBf16 ? 2 : 4;
};

// 32 bytes, not kept in L1 (each byte of a row is read once).
__device__ __forceinline__ void ld_row32(const void *p, uint32_t (&r)[8])
{
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p)
                 : "memory");
}

// 32 bytes that other warps of the SM read as well.
__device__ __forceinline__ void ld_kept32(const void *p, uint32_t (&r)[8])
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p)
                 : "memory");
}

__device__ __forceinline__ void st_row32(void *p, const uint32_t (&r)[8])
{
    asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Pairs of FP32 values in one 64-bit register: the packed product and
// multiply-add round each half as the scalar ones do.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float lo, float hi)
{
    F2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void f2_split(F2 v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b)
{
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c)
{
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b)
{
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// A word of two BF16 values as an FP32 pair.
__device__ __forceinline__ F2 f2_bf16(uint32_t w)
{
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Sixteen values as loaded: one 32-byte access in BF16, two in FP32.
template <int DT>
struct Raw16 {
    static constexpr int kParts = DT == kBf16 ? 1 : 2;
    uint32_t r[kParts][8];

    template <bool KEPT = false>
    __device__ __forceinline__ void load(const char *p, bool inside)
    {
#pragma unroll
        for (int l = 0; l < kParts; ++l) {
            if (inside) {
                if (KEPT)
                    ld_kept32(p + 32 * l, r[l]);
                else
                    ld_row32(p + 32 * l, r[l]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[l][i] = 0;
            }
        }
    }

    __device__ __forceinline__ float at(int i) const
    {
        if (DT == kBf16) {
            const uint32_t w = r[0][i >> 1];
            return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
        }
        return __uint_as_float(r[(i >> 3) & (kParts - 1)][i & 7]);
    }

    // values 2i and 2i + 1
    __device__ __forceinline__ F2 pair(int i) const
    {
        if constexpr (DT == kBf16)
            return f2_bf16(r[0][i]);
        else
            return f2(at(2 * i), at(2 * i + 1));
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// Sixteen FP32 values stored as DT (BF16: rounded to nearest even).
template <int DT>
__device__ __forceinline__ void store16(char *p, const float (&v)[kLaneVals])
{
    uint32_t w[8];
    if (DT == kBf16) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        st_row32(p, w);
    } else {
#pragma unroll
        for (int l = 0; l < 2; ++l) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = __float_as_uint(v[8 * l + i]);
            st_row32(p + 32 * l, w);
        }
    }
}

// Two FP32 products in one instruction (the packed form has twice the scalar rate).
__device__ __forceinline__ void mul2(float &d0, float &d1, float a0, float a1, float b0, float b1)
{
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// max(|a|, |b|, |c|); a NaN among them gives NaN.
__device__ __forceinline__ float max_abs3(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Bit pattern of the largest magnitude of a lane's sixteen values.  Patterns of
// magnitudes order like the values, and a NaN's is above the infinity's.
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[kLaneVals])
{
    float m = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i + 1 < kLaneVals; i += 2)
        m = max_abs3(m, v[i], v[i + 1]);
    return __float_as_uint(max_abs3(m, v[kLaneVals - 1], v[kLaneVals - 1]));
}

// The same from the values as loaded; BF16 pairs are compared two at a time.
template <int DT>
__device__ __forceinline__ uint32_t amax_bits(const Raw16<DT> &x)
{
    if constexpr (DT == kBf16) {
        uint32_t m = x.r[0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i)
            asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x.r[0][i]));
        m &= 0x7FFF7FFFu;
        return max(m << 16, m & 0xFFFF0000u);
    } else {
        float v[kLaneVals];
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i)
            v[i] = x.at(i);
        return amax_bits(v);
    }
}

// Two FP32 values -> two E4M3 codes (lo in the low byte), nearest-even, saturating.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Eight FP32 values -> eight E2M1 codes, value i in nibble i, nearest-even, saturating.
__device__ __forceinline__ uint32_t e2m1_word(const float *v)
{
    uint32_t d;
    asm("{\n\t"
        ".reg .b8 q0, q1, q2, q3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 q0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 q1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 q2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 q3, %8, %7;\n\t"
        "mov.b32 %0, {q0, q1, q2, q3};\n\t"
        "}"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

// A lane's sixteen encoded values and the scale word of its K-tile.
template <int FMT>
struct Codes16 {
    static constexpr int kWords = FMT == kMxfp8 ? 4 : 2;
    uint32_t w[kWords];
    uint32_t scode;  // scale code of this lane's block
};

// Encode a warp's chunk whose lanes' largest magnitudes are `amax` (every lane of
// the warp calls it; lanes outside the row hold zeros).
template <int FMT>
__device__ __forceinline__ Codes16<FMT> mx_encode(const float (&v)[kLaneVals], uint32_t amax)
{
    constexpr int kEMax = FMT == kMxfp8 ? 8 : 2;
    Codes16<FMT> c;
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    const bool nonfinite = amax >= 0x7F800000u;
    const int scode = amax == 0 ? 127 : max(static_cast<int>(amax >> 23) - kEMax, 0);
    const float mul = __uint_as_float(static_cast<uint32_t>(254 - scode) << 23);  // 2^(127 - scode), exact products
    c.scode = nonfinite ? 255u : static_cast<uint32_t>(scode);
    float t[kLaneVals];
#pragma unroll
    for (int i = 0; i < kLaneVals; i += 2)
        mul2(t[i], t[i + 1], v[i], v[i + 1], mul, mul);
    if (FMT == kMxfp8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = e4m3_pair(t[4 * i], t[4 * i + 1]);
            const uint32_t hi = e4m3_pair(t[4 * i + 2], t[4 * i + 3]);
            c.w[i] = nonfinite ? 0u : (lo | (hi << 16));
        }
    } else {
        c.w[0] = nonfinite ? 0u : e2m1_word(t);
        c.w[Codes16<FMT>::kWords - 1] = nonfinite ? 0u : e2m1_word(t + 8);
    }
    return c;
}

template <int FMT>
__device__ __forceinline__ Codes16<FMT> mx_encode(const float (&v)[kLaneVals])
{
    return mx_encode<FMT>(v, amax_bits(v));
}

// The four scale codes of this lane's K-tile in one word (block c in byte c).
__device__ __forceinline__ uint32_t tile_scale_word(uint32_t scode, int lane)
{
    uint32_t w = scode << (8 * ((lane >> 1) & 3));
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, 2);
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, 4);
    return w;
}

// Codes of a lane at value k of a row (FMT bytes per value).
template <int FMT>
__device__ __forceinline__ void store_codes(uint8_t *row_codes, int64_t k, const Codes16<FMT> &c)
{
    if (FMT == kMxfp8)
        *reinterpret_cast<uint4 *>(row_codes + k) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
    else
        *reinterpret_cast<uint2 *>(row_codes + (k >> 1)) = make_uint2(c.w[0], c.w[1]);
}

// How a scale tensor is laid out.
constexpr int kScaleBytes = 0;  // row-major, written byte by byte (K not a multiple of 128)
constexpr int kScaleWords = 1;  // row-major, one word per K-tile
constexpr int kScaleTiled = 2;  // the 512-byte tile layout

// Byte offset of the four scales of (row, K-tile kt) in the tile layout.
__device__ __forceinline__ int64_t tile_scale_offset(int64_t row, int64_t kt, int64_t num_kt)
{
    return ((row >> 7) * num_kt + kt) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Scales of a warp's chunk that starts at value k0 of `row` (every lane calls it).
__device__ __forceinline__ void store_scales(uint8_t *scales, int mode, int64_t row, int64_t k0, int64_t K, int lane,
                                             uint32_t scode)
{
    const int64_t k = k0 + lane * kLaneVals;
    if (mode == kScaleBytes) {
        if ((lane & 1) == 0 && k < K)
            scales[row * (K >> 5) + (k >> 5)] = static_cast<uint8_t>(scode);
        return;
    }
    const uint32_t w = tile_scale_word(scode, lane);
    if ((lane & 7) == 0 && k < K) {
        const int64_t at = mode == kScaleTiled ? tile_scale_offset(row, k >> 7, K >> 7) : row * (K >> 5) + (k >> 5);
        *reinterpret_cast<uint32_t *>(scales + at) = w;
    }
}

// Tile layout: the rows from `rows` up to the next multiple of 128 hold code 127
// (x1.0).  Called by every thread of a grid of `nthreads` threads.
__device__ __forceinline__ void pad_tiled_scales(uint8_t *scales, int64_t rows, int64_t K, int64_t tid,
                                                 int64_t nthreads)
{
    const int64_t num_kt = K >> 7;
    const int64_t n = (((rows + 127) & ~int64_t(127)) - rows) * num_kt;
    for (int64_t i = tid; i < n; i += nthreads)
        *reinterpret_cast<uint32_t *>(scales + tile_scale_offset(rows + i / num_kt, i % num_kt, num_kt)) = 0x7F7F7F7Fu;
}

// Sixteen MXFP8 codes times their block's scale, as pairs.  Code 0xFF of the scale is
// NaN.  The product of an E4M3 value and a power of two is exact in FP32 unless it
// underflows past the smallest subnormal.
__device__ __forceinline__ void decode_e4m3(const uint4 q, uint32_t scode, F2 (&v)[kLaneVals / 2])
{
    // 2^(scode - 127): scode 0 is the subnormal 2^-127
    const float s = scode == 255u ? __uint_as_float(0x7FC00000u)
                                  : __uint_as_float(scode == 0 ? 0x00400000u : scode << 23);
    const F2 s2 = f2(s, s);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint16_t pair = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        uint32_t h2;  // two halves; every E4M3 value is a half
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(pair));
        float lo, hi;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "r"(h2));
        v[i] = f2_mul(f2(lo, hi), s2);
    }
}

// The sixteen values of eight pairs.
__device__ __forceinline__ void f2_unpack(const F2 (&p)[kLaneVals / 2], float (&v)[kLaneVals])
{
#pragma unroll
    for (int i = 0; i < kLaneVals / 2; ++i)
        f2_split(p[i], v[2 * i], v[2 * i + 1]);
}

// A warp's walk over the 512-value chunks of a matrix's rows, every `step`-th chunk
// from `first` on: one division at the start, additions from then on.
struct ChunkWalk {
    int64_t row;
    int chunk, per_row;
    int64_t row_step;
    int chunk_step;

    __device__ __forceinline__ ChunkWalk(int64_t row_len, int64_t first, int64_t step)
    {
        per_row = static_cast<int>((row_len + kWarpVals - 1) / kWarpVals);
        row = first / per_row;
        chunk = static_cast<int>(first - row * per_row);
        row_step = step / per_row;
        chunk_step = static_cast<int>(step - row_step * per_row);
    }
    __device__ __forceinline__ void next()
    {
        row += row_step;
        chunk += chunk_step;
        if (chunk >= per_row) {
            chunk -= per_row;
            ++row;
        }
    }
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

}  // namespace mxg
