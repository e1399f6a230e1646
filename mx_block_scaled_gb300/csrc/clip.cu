// clip.cu -- the global norm of many gradients, and the gradients clipped to it.
//
//   norm = sqrt(sum over all tensors of g^2);  out = g * min(1, max_norm / (norm + 1e-6))
//
// All tensors of a call (a thousand a launch) are one list of chunks of 4096 values;
// a block takes a contiguous part of it, so that the tensors' number and sizes do not
// matter.  The table of tensors is a kernel parameter: no copy to the device, and a
// captured call keeps its own.  Squares are summed in FP32 16 or 32 at a time where
// that sum keeps its precision, else in FP64, and on in FP64; a block leaves
// one partial sum, and every block of the second kernel adds those in the same order.
// That kernel walks its part backwards: what the first read last is still in L2.
#include "mx_block.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kChunk = static_cast<int64_t>(kThreads) * kLaneVals;
constexpr int kBlocksPerSm = 4;

template <int N>
struct Table {
    GradTensor t[N];
    uint32_t end[N];  // chunks up to and with tensor i
    int n;
    uint32_t chunks;
};

// A thread's values of a tensor come eight at a time, a block's next to each other: a
// BF16 load is 16 bytes, an FP32 one 32, and a warp's accesses are consecutive whatever
// the two types.
constexpr int kVals = 8;
constexpr int kSteps = static_cast<int>(kChunk / (kThreads * kVals));  // of a chunk
static_assert(kSteps == 2, "a thread takes two runs of eight values of a chunk");

// Part of a tensor that is a block's: chunks [from, to) counted in the tensor.
struct Part {
    int i;
    int64_t from, to;
};

// A block's walk over the tensors of its chunks [c0, c1), forwards or backwards.
template <int N, bool BACKWARDS>
struct Walk {
    const Table<N> &table;
    uint32_t c0, c1;
    int i;

    __device__ __forceinline__ Walk(const Table<N> &t, uint32_t from, uint32_t to) : table(t), c0(from), c1(to)
    {
        const uint32_t chunk = BACKWARDS ? to - 1 : from;
        int lo = 0, hi = t.n - 1;  // the first tensor that ends past the chunk
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (t.end[mid] > chunk)
                hi = mid;
            else
                lo = mid + 1;
        }
        i = lo;
    }
    __device__ __forceinline__ bool next(Part &p)
    {
        if (c0 >= c1)
            return false;
        uint32_t begin = i > 0 ? table.end[i - 1] : 0;
        if (BACKWARDS) {
            while (begin >= c1)  // (tensors without values)
                begin = --i > 0 ? table.end[i - 1] : 0;
            const uint32_t first = begin > c0 ? begin : c0;
            p = {i, first - begin, c1 - begin};
            c1 = first;
        } else {
            while (table.end[i] <= c0)
                begin = table.end[i++];
            const uint32_t last = table.end[i] < c1 ? table.end[i] : c1;
            p = {i, c0 - begin, last - begin};
            c0 = last;
        }
        return true;
    }
};

// Eight values as they are in memory; zeros past the tensor's end.
struct Values {
    uint32_t r[8];

    template <bool BF16>
    __device__ __forceinline__ void load(const GradTensor &t, int64_t at)
    {
        const int64_t left = t.n - at;
        if (left >= kVals && (t.flags & kGradSrcVector)) {
            if constexpr (BF16)
                asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                             : "l"(static_cast<const char *>(t.src) + at * 2)
                             : "memory");
            else
                ld_row32(static_cast<const char *>(t.src) + at * 4, r);
            return;
        }
#pragma unroll
        for (int i = 0; i < (BF16 ? 4 : 8); ++i)
            r[i] = 0;
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            if (i < left) {
                if constexpr (BF16)
                    r[i >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t *>(t.src)[at + i]) << (16 * (i & 1));
                else
                    r[i] = static_cast<const uint32_t *>(t.src)[at + i];
            }
    }
    template <bool BF16>
    __device__ __forceinline__ F2 pair(int i) const
    {
        if constexpr (BF16)
            return f2_bf16(r[i]);
        else
            return f2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
    }
};

template <bool BF16>
__device__ __forceinline__ void store_values(const GradTensor &t, int64_t at, const float (&v)[kVals])
{
    const int64_t left = t.n - at;
    if (left >= kVals && (t.flags & kGradDstVector)) {
        if constexpr (BF16) {
            *reinterpret_cast<uint4 *>(static_cast<char *>(t.dst) + at * 2) = make_uint4(
                pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < kVals; ++i)
                w[i] = __float_as_uint(v[i]);
            st_row32(static_cast<char *>(t.dst) + at * 4, w);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kVals; ++i)
        if (i < left) {
            if constexpr (BF16)
                static_cast<__nv_bfloat16 *>(t.dst)[at + i] = __float2bfloat16_rn(v[i]);
            else
                static_cast<float *>(t.dst)[at + i] = v[i];
        }
}

__device__ __forceinline__ double warp_sum64(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ double block_sum64(double v, double *part)
{
    v = warp_sum64(v);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        s += part[w];
    return s;
}

// Sums of squares between these keep FP32's precision: none overflowed, and what
// underflowed is below 2^-33 of the sum.
constexpr float kSumLeast = 7.7e-34f, kSumMost = 1.2e30f;  // about 2^-110 and 2^100

// Runs of eight values that a thread has in flight: 64 bytes.
template <bool BF16>
constexpr int kAhead = BF16 ? 4 : 2;

// The sum of the squares of a block's part of a tensor, added to this thread's.
template <bool BF16>
__device__ __forceinline__ void sum_part(const GradTensor &t, const Part &p, double &sum)
{
    constexpr int U = kAhead<BF16>;
    const int64_t last = p.to * kSteps;
    int64_t step = p.from * kSteps;  // runs of a thread, counted in the tensor
    Values next[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        next[u].template load<BF16>(t, step + u < last ? ((step + u) * kThreads + threadIdx.x) * kVals : t.n);
    for (; step < last; step += U) {
        Values v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = next[u];
        if (step + U < last)
#pragma unroll
            for (int u = 0; u < U; ++u)
                next[u].template load<BF16>(t, step + U + u < last ? ((step + U + u) * kThreads + threadIdx.x) * kVals
                                                                   : t.n);
        F2 s2 = f2(0.0f, 0.0f);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < kVals / 2; ++i)
                s2 = f2_fma(v[u].template pair<BF16>(i), v[u].template pair<BF16>(i), s2);
        float a, b;
        f2_split(s2, a, b);
        const float s = a + b;
        if (s > kSumLeast && s < kSumMost) {
            sum += s;
        } else {
            uint32_t any = 0;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < (BF16 ? 4 : 8); ++i)
                    any |= v[u].r[i] & (BF16 ? 0x7FFF7FFFu : 0x7FFFFFFFu);
            if (any != 0)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < kVals / 2; ++i) {
                        f2_split(v[u].template pair<BF16>(i), a, b);
                        sum += static_cast<double>(a) * a + static_cast<double>(b) * b;
                    }
        }
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    grad_norm_kernel(const __grid_constant__ Table<N> table, double *partial)
{
    __shared__ double part[kWarps];
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t c0 = static_cast<uint32_t>(static_cast<uint64_t>(table.chunks) * blockIdx.x / gridDim.x);
    const uint32_t c1 = static_cast<uint32_t>(static_cast<uint64_t>(table.chunks) * (blockIdx.x + 1) / gridDim.x);
    double sum = 0.0;
    if (c0 < c1) {
        Walk<N, false> walk(table, c0, c1);
        for (Part p; walk.next(p);) {
            if (table.t[p.i].flags & kGradSrcBf16)
                sum_part<true>(table.t[p.i], p, sum);
            else
                sum_part<false>(table.t[p.i], p, sum);
        }
    }
    sum = block_sum64(sum, part);
    if (threadIdx.x == 0)
        partial[blockIdx.x] = sum;
}

// The sum of all squares from the blocks' sums.
__device__ __forceinline__ double total_of(const double *partial, int n, double *part)
{
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads)
        s += __ldcg(partial + i);
    return block_sum64(s, part);
}

// Norm and factor in FP32 where the sum is well inside its range: FP64's root and
// quotient take a microsecond here.
constexpr double kTotalLeast = 1e-30, kTotalMost = 1e30;

__device__ __forceinline__ float norm_of(double total)
{
    return total > kTotalLeast && total < kTotalMost ? sqrtf(static_cast<float>(total))
                                                     : static_cast<float>(sqrt(total));
}

__device__ __forceinline__ float factor_of(double total, float max_norm)
{
    const float f = total > kTotalLeast && total < kTotalMost
                        ? max_norm / (sqrtf(static_cast<float>(total)) + 1e-6f)
                        : static_cast<float>(static_cast<double>(max_norm) / (sqrt(total) + 1e-6));
    return f >= 1.0f ? 1.0f : f;  // a norm of NaN gives NaN
}

__global__ void __launch_bounds__(kThreads) grad_norm_finish_kernel(const double *partial, int n, float *norm)
{
    __shared__ double part[kWarps];
    griddep_launch_dependents();
    griddep_wait();
    const double total = total_of(partial, n, part);
    if (threadIdx.x == 0)
        *norm = norm_of(total);
}

// A block's part of a tensor times the factor, from its end to its start.
template <bool SRC, bool DST>
__device__ __forceinline__ void clip_part(const GradTensor &t, const Part &p, float factor)
{
    constexpr int U = kAhead<SRC>;
    const int64_t first = p.from * kSteps;
    int64_t step = p.to * kSteps;  // one past the run that is next
    auto at = [&](int64_t run) { return (run * kThreads + threadIdx.x) * kVals; };
    Values next[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        next[u].template load<SRC>(t, step - 1 - u >= first ? at(step - 1 - u) : t.n);
    const F2 f = f2(factor, factor);
    for (; step > first; step -= U) {
        Values v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = next[u];
        if (step - U > first)
#pragma unroll
            for (int u = 0; u < U; ++u)
                next[u].template load<SRC>(t, step - U - 1 - u >= first ? at(step - U - 1 - u) : t.n);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (step - 1 - u < first)
                break;
            float o[kVals];
#pragma unroll
            for (int i = 0; i < kVals / 2; ++i)
                f2_split(f2_mul(v[u].template pair<SRC>(i), f), o[2 * i], o[2 * i + 1]);
            store_values<DST>(t, at(step - 1 - u), o);
        }
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    grad_clip_kernel(const __grid_constant__ Table<N> table, const double *partial, int n, float max_norm, float *norm)
{
    __shared__ double part[kWarps];
    __shared__ float block_factor;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t c0 = static_cast<uint32_t>(static_cast<uint64_t>(table.chunks) * blockIdx.x / gridDim.x);
    const uint32_t c1 = static_cast<uint32_t>(static_cast<uint64_t>(table.chunks) * (blockIdx.x + 1) / gridDim.x);
    const double total = total_of(partial, n, part);
    if (threadIdx.x == 0) {
        block_factor = factor_of(total, max_norm);
        if (norm && blockIdx.x == 0)
            *norm = norm_of(total);
    }
    __syncthreads();
    const float factor = block_factor;
    if (c0 >= c1)
        return;
    Walk<N, true> walk(table, c0, c1);
    for (Part p; walk.next(p);) {
        const GradTensor &t = table.t[p.i];
        if (factor == 1.0f && t.src == t.dst)
            continue;  // what stays as it is need not be written
        if (t.flags & kGradSrcBf16) {
            if (t.flags & kGradDstBf16)
                clip_part<true, true>(t, p, factor);
            else
                clip_part<true, false>(t, p, factor);
        } else {
            if (t.flags & kGradDstBf16)
                clip_part<false, true>(t, p, factor);
            else
                clip_part<false, false>(t, p, factor);
        }
    }
}

template <int N>
cudaError_t launch_tables(const GradTensor *tensors, int64_t n, int num_sms, bool clip, double *partial, int parts,
                          float max_norm, float *norm, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    for (int64_t at = 0; at < n; at += N) {
        Table<N> table;
        table.n = static_cast<int>(n - at < N ? n - at : N);
        uint32_t chunks = 0;
        for (int i = 0; i < table.n; ++i) {
            table.t[i] = tensors[at + i];
            chunks += static_cast<uint32_t>((tensors[at + i].n + kChunk - 1) / kChunk);
            table.end[i] = chunks;
        }
        table.chunks = chunks;
        const unsigned blocks = grad_blocks(num_sms);
        const cudaLaunchConfig_t cfg = row_launch(blocks, kThreads, 0, s, attr);
        const cudaError_t e =
            clip ? cudaLaunchKernelEx(&cfg, grad_clip_kernel<N>, table, static_cast<const double *>(partial), parts,
                                      max_norm, at == 0 ? norm : nullptr)
                 : cudaLaunchKernelEx(&cfg, grad_norm_kernel<N>, table, partial + at / N * blocks);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

// Few tensors take a short table: a launch copies its parameters.
constexpr int kTables[3] = {32, 256, 896};

int table_size(int64_t n) { return n <= kTables[0] ? kTables[0] : n <= kTables[1] ? kTables[1] : kTables[2]; }

cudaError_t launch_any(const GradTensor *tensors, int64_t n, int num_sms, bool clip, double *partial, int parts,
                       float max_norm, float *norm, cudaStream_t s)
{
    const int size = table_size(n);
    return size == kTables[0]   ? launch_tables<kTables[0]>(tensors, n, num_sms, clip, partial, parts, max_norm, norm, s)
           : size == kTables[1] ? launch_tables<kTables[1]>(tensors, n, num_sms, clip, partial, parts, max_norm, norm, s)
                                : launch_tables<kTables[2]>(tensors, n, num_sms, clip, partial, parts, max_norm, norm, s);
}

int launches(int64_t n) { return static_cast<int>((n + table_size(n) - 1) / table_size(n)); }  // none for n = 0

}  // namespace

unsigned grad_blocks(int num_sms)
{
    return static_cast<unsigned>((num_sms < kGradSms ? num_sms : kGradSms) * kBlocksPerSm);
}

size_t grad_workspace(int64_t n) { return static_cast<size_t>(launches(n)) * grad_blocks(kGradSms) * sizeof(double); }

// Chunks of 4096 values of a launch are numbered in 32 bits.
bool grads_fit(const GradTensor *tensors, int64_t n)
{
    const int size = n > 0 ? table_size(n) : 1;
    int64_t chunks = 0;
    for (int64_t i = 0; i < n; ++i) {
        chunks = (i % size == 0 ? 0 : chunks) + (tensors[i].n + kChunk - 1) / kChunk;
        if (chunks > 0x7FFFFFFF)
            return false;
    }
    return true;
}

cudaError_t launch_grad_norm(const GradTensor *tensors, int64_t n, double *partial, float *norm, int num_sms,
                             cudaStream_t s)
{
    cudaError_t e = launch_any(tensors, n, num_sms, false, partial, 0, 0.0f, nullptr, s);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = row_launch(1, kThreads, 0, s, attr);
    return cudaLaunchKernelEx(&cfg, grad_norm_finish_kernel, static_cast<const double *>(partial),
                              launches(n) * static_cast<int>(grad_blocks(num_sms)), norm);
}

cudaError_t launch_clip_grads(const GradTensor *tensors, int64_t n, double *partial, float max_norm, float *norm,
                              int num_sms, cudaStream_t s)
{
    if (n == 0)
        return launch_grad_norm(tensors, n, partial, norm, num_sms, s);
    const cudaError_t e = launch_any(tensors, n, num_sms, false, partial, 0, 0.0f, nullptr, s);
    return e != cudaSuccess ? e
                            : launch_any(tensors, n, num_sms, true, partial,
                                         launches(n) * static_cast<int>(grad_blocks(num_sms)), max_norm, norm, s);
}

}  // namespace mxg
