// clip.cu -- the global norm of many gradients, and the gradients clipped to it.
//
//   norm = sqrt(sum over all tensors of g^2);  out = g * min(1, max_norm / (norm + 1e-6))
//
// All tensors of a call (a thousand a launch) are one list of chunks of 4096 values;
// a block takes a contiguous part of it, so that the tensors' number and sizes do not
// matter.  The table of tensors is a kernel parameter: no copy to the device, and a
// captured call keeps its own.  Squares are summed in FP32 sixteen at a time where
// that sum keeps its precision, else from FP64 squares, and on in FP64; a block leaves
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

// A block's walk over its part of the chunks.
template <int N>
struct Walk {
    const Table<N> &table;
    int i;             // tensor
    uint32_t first;    // its first chunk

    __device__ __forceinline__ Walk(const Table<N> &t, uint32_t chunk) : table(t)
    {
        int lo = 0, hi = t.n - 1;  // the first tensor that ends past the chunk
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (t.end[mid] > chunk)
                hi = mid;
            else
                lo = mid + 1;
        }
        i = lo;
        first = i > 0 ? t.end[i - 1] : 0;
    }
    __device__ __forceinline__ void to(uint32_t chunk)  // a neighbour of the last one
    {
        while (chunk >= table.end[i])
            first = table.end[i++];
        while (chunk < first) {
            --i;
            first = i > 0 ? table.end[i - 1] : 0;
        }
    }
    // Values of this thread in the chunk: from, and how many (at most sixteen).
    __device__ __forceinline__ int64_t at(uint32_t chunk, int &count) const
    {
        const int64_t from = static_cast<int64_t>(chunk - first) * kChunk + threadIdx.x * kLaneVals;
        const int64_t left = table.t[i].n - from;
        count = left >= kLaneVals ? kLaneVals : left > 0 ? static_cast<int>(left) : 0;
        return from;
    }
};

// Sixteen values of a tensor as FP32 (zeros past `count`).
__device__ __forceinline__ void load_values(const GradTensor &t, int64_t from, int count, float (&v)[kLaneVals])
{
    if (count == kLaneVals && (t.flags & kGradSrcVector)) {
        if (t.flags & kGradSrcBf16) {
            Raw16<kBf16> x;
            x.load(static_cast<const char *>(t.src) + from * 2, true);
#pragma unroll
            for (int i = 0; i < kLaneVals; ++i)
                v[i] = x.at(i);
        } else {
            Raw16<kF32> x;
            x.load(static_cast<const char *>(t.src) + from * 4, true);
#pragma unroll
            for (int i = 0; i < kLaneVals; ++i)
                v[i] = x.at(i);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i) {
        v[i] = 0.0f;
        if (i < count)
            v[i] = (t.flags & kGradSrcBf16)
                       ? __bfloat162float(static_cast<const __nv_bfloat16 *>(t.src)[from + i])
                       : static_cast<const float *>(t.src)[from + i];
    }
}

__device__ __forceinline__ void store_values(const GradTensor &t, int64_t from, int count, const float (&v)[kLaneVals])
{
    if (count == kLaneVals && (t.flags & kGradDstVector)) {
        if (t.flags & kGradDstBf16)
            store16<kBf16>(static_cast<char *>(t.dst) + from * 2, v);
        else
            store16<kF32>(static_cast<char *>(t.dst) + from * 4, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i)
        if (i < count) {
            if (t.flags & kGradDstBf16)
                static_cast<__nv_bfloat16 *>(t.dst)[from + i] = __float2bfloat16_rn(v[i]);
            else
                static_cast<float *>(t.dst)[from + i] = v[i];
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

// Sums of sixteen squares between these keep FP32's precision: none overflowed, and
// what underflowed is below 2^-35 of the sum.
constexpr float kSumLeast = 7.7e-34f, kSumMost = 1.2e30f;  // about 2^-110 and 2^100
constexpr int kWindow = 4;                                 // FP32 sums that are added up before they go to FP64

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
    float window = 0.0f;
    int in_window = 0;
    if (c0 < c1) {
        Walk<N> walk(table, c0);
        float next[kLaneVals];
        int count;
        int64_t from = walk.at(c0, count);
        load_values(table.t[walk.i], from, count, next);
        for (uint32_t c = c0; c < c1; ++c) {
            float v[kLaneVals];
#pragma unroll
            for (int i = 0; i < kLaneVals; ++i)
                v[i] = next[i];
            if (c + 1 < c1) {
                walk.to(c + 1);
                from = walk.at(c + 1, count);
                load_values(table.t[walk.i], from, count, next);
            }
            F2 s2 = f2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < kLaneVals; i += 2)
                s2 = f2_fma(f2(v[i], v[i + 1]), f2(v[i], v[i + 1]), s2);
            float a, b;
            f2_split(s2, a, b);
            const float s = a + b;
            if (s > kSumLeast && s < kSumMost) {
                window += s;
                if (++in_window == kWindow) {
                    sum += window;
                    window = 0.0f;
                    in_window = 0;
                }
            } else {
                uint32_t any = 0;
#pragma unroll
                for (int i = 0; i < kLaneVals; ++i)
                    any |= __float_as_uint(v[i]) & 0x7FFFFFFFu;
                if (any != 0)
#pragma unroll 1
                    for (int i = 0; i < kLaneVals; ++i) {
                        const double d = v[i];
                        sum += d * d;
                    }
            }
        }
    }
    sum = block_sum64(sum + window, part);
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
    Walk<N> walk(table, c1 - 1);
    float next[kLaneVals];
    int count;
    int64_t from = walk.at(c1 - 1, count);
    load_values(table.t[walk.i], from, count, next);
    for (uint32_t c = c1; c-- > c0;) {
        const int64_t at = from;
        const int had = count;
        const GradTensor &t = table.t[walk.i];
        float v[kLaneVals];
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i)
            v[i] = next[i] * factor;
        if (c > c0) {
            walk.to(c - 1);
            from = walk.at(c - 1, count);
            load_values(table.t[walk.i], from, count, next);
        }
        if (factor != 1.0f || t.src != t.dst)  // what stays as it is need not be written
            store_values(t, at, had, v);
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
