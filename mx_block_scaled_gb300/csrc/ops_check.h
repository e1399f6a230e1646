// ops_check.h -- argument checks that the row operators' entry points share.
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include <cuda_runtime.h>

#include "mxgemm.h"

namespace mxg {

// Kernels that a device is prepared for (shared memory, cluster sizes) before their first launch.  Each family by itself:
// a call prepares, and fails for, no other's.
enum Family { kNormGradient, kEmbedGradient, kHeads, kUnprepared };

// The current device's SM count, with the family's kernels prepared on it (ops.cu).
int ops_device(int *num_sms, Family family = kUnprepared);

inline int status_of(cudaError_t e) { return e == cudaSuccess ? MXGEMM_OK : MXGEMM_ERR_CUDA; }

inline bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int64_t kMaxRows = (1ll << 31) - 1;
constexpr int64_t kMaxCols = 1ll << 30;

inline bool known_dtype(int d) { return d == MXGEMM_IN_F32 || d == MXGEMM_IN_BF16; }
inline int64_t elem_bytes(int d) { return d == MXGEMM_IN_BF16 ? 2 : 4; }
inline const char *bytes(const void *p) { return static_cast<const char *>(p); }

// A strided input matrix: NULL passes; rows start on 32-byte boundaries and do
// not overlap (a stride of at least the row, or a single row).
inline bool rows_shape_ok(const void *p, int64_t stride, int64_t rows, int64_t cols)
{
    return p == nullptr || rows == 1 || (stride >= cols && stride <= (1ll << 40));
}
inline bool rows_align_ok(const void *p, int64_t stride, int64_t rows, int64_t elem)
{
    return p == nullptr || (aligned(p, 32) && (rows == 1 || stride * elem % 32 == 0));
}

// Bytes of a matrix, from its first to its last; p NULL for one that there is not.
struct Span {
    const void *p;
    int64_t rows, stride, row;
};
inline Span dense(const void *p, int64_t rows, int64_t row) { return {p, rows, row, row}; }
inline Span flat(const void *p, int64_t n) { return {p, 1, n, n}; }

inline bool apart(const Span &a, const Span &b)
{
    if (!a.p || !b.p)
        return true;
    using Wide = unsigned __int128;  // no size that the other checks pass overflows it
    const Wide a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 + static_cast<Wide>(a.rows - 1) * a.stride + a.row <= b0 ||
           b0 + static_cast<Wide>(b.rows - 1) * b.stride + b.row <= a0;
}

// An output, and the inputs (bit i: input i) that it may be itself: whole and dense,
// where the thread that writes a value is the one that read it, and had read it before.
struct Output {
    Span at;
    unsigned over = 0;

    bool is(const Span &in) const
    {
        return at.p == in.p && at.rows == in.rows && at.row == in.row && (in.rows == 1 || in.stride == in.row);
    }
};

// No output touches a byte of an input, apart from those that it may be, nor of another
// output: blocks read inputs while others write.
inline bool outputs_apart(std::initializer_list<Output> outs, std::initializer_list<Span> ins)
{
    for (const Output *o = outs.begin(); o != outs.end(); ++o) {
        unsigned bit = 1;
        for (const Span &in : ins) {
            if (!apart(o->at, in) && !((o->over & bit) && o->is(in)))
                return false;
            bit <<= 1;
        }
        for (const Output *other = outs.begin(); other != o; ++other)
            if (!apart(o->at, other->at))
                return false;
    }
    return true;
}

}  // namespace mxg
