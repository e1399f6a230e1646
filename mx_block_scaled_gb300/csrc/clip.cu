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
//
// Bound by HBM: 872 M BF16 values summed in 247 us (7.1 TB/s), scaled into FP32 in 854 more
// (6.1 TB/s); 42 M FP32 values of 448 tensors 30 and 51 us.  Four million BF16 values take
// 8.0 us, one million 5.6, two launches' latency.
#include <algorithm>

#include "mx_block.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kChunk = static_cast<int64_t>(kThreads) * kLaneVals;
// A block reads a contiguous part, so more of them are more places of HBM that are read at once: 872 M BF16 values
// summed in 302 us with two a multiprocessor, 255 with three, 248 with four, 415 with six.
constexpr int kBlocksPerSm = 4;

constexpr int kMostBlocks = kGradSms * kBlocksPerSm;

template <int N>
struct Table {
    GradTensor t[N];
    uint32_t end[N];                      // chunks up to and with tensor i
    uint16_t start[kMostBlocks + 1];      // the tensor of a block's first chunk, and of the last chunk
    uint32_t chunks;

    __device__ __forceinline__ uint32_t chunk_of(uint32_t block) const  // a block's first chunk
    {
        return static_cast<uint32_t>(static_cast<uint64_t>(chunks) * block / gridDim.x);
    }
};

// A thread's values of a tensor come eight at a time, a block's next to each other: a
// BF16 load is 16 bytes, an FP32 one 32, and a warp's accesses are consecutive whatever
// the two types.
constexpr int kVals = 8;
constexpr int kSteps = static_cast<int>(kChunk / (kThreads * kVals));  // of a chunk
static_assert(kSteps == 2, "a thread takes two runs of eight values of a chunk");

// Part of a tensor that is a block's: chunks [from, to) counted in the tensor.
struct Part {
    int i = 0;
    int64_t from = 0, to = 0;
};

// A tensor of the table.
struct Tensor {
    const void *src;
    void *dst;
    int64_t n;
    uint32_t flags;

    __device__ __forceinline__ explicit Tensor(const GradTensor &t)
        : src(t.src), dst(t.dst), n(t.n_flags >> kGradFlagBits), flags(static_cast<uint32_t>(t.n_flags) & ((1u << kGradFlagBits) - 1))
    {
    }
};

// A block's walk over the tensors of its chunks [c0, c1), forwards or backwards (from the tensor of the next block's
// first chunk on).
template <int N, bool BACKWARDS>
struct Walk {
    const Table<N> &table;
    uint32_t c0, c1;
    int i;

    __device__ __forceinline__ explicit Walk(const Table<N> &t)
        : table(t), c0(t.chunk_of(blockIdx.x)), c1(t.chunk_of(blockIdx.x + 1)), i(t.start[blockIdx.x + BACKWARDS])
    {
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

// Eight values as they are in memory.
template <bool BF16>
struct Values {
    static constexpr int kWords = BF16 ? 4 : 8;
    uint32_t r[kWords];

    __device__ __forceinline__ void load(const void *p)
    {
        if constexpr (BF16)
            asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                         : "l"(p)
                         : "memory");
        else
            ld_row32(p, r);
    }
    // the first `left` of them (any number), one by one; zeros after
    __device__ __forceinline__ void load_some(const void *p, int64_t left)
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            r[i] = 0;
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            if (i < left) {
                if constexpr (BF16)
                    r[i >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << (16 * (i & 1));
                else
                    r[i] = static_cast<const uint32_t *>(p)[i];
            }
    }
    __device__ __forceinline__ F2 pair(int i) const
    {
        if constexpr (BF16)
            return f2_bf16(r[i]);
        else
            return f2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
    }
};

// Eight FP32 values as eight of the output's, and the first `left` of them.
template <bool BF16>
__device__ __forceinline__ void store_values(void *p, const float (&v)[kVals])
{
    if constexpr (BF16) {
        *static_cast<uint4 *>(p) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            w[i] = __float_as_uint(v[i]);
        st_row32(p, w);
    }
}

template <bool BF16>
__device__ __forceinline__ void store_some(void *p, int64_t left, const float (&v)[kVals])
{
#pragma unroll
    for (int i = 0; i < kVals; ++i)
        if (i < left) {
            if constexpr (BF16)
                static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v[i]);
            else
                static_cast<float *>(p)[i] = v[i];
        }
}

__device__ __forceinline__ double warp_sum64(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The sum over the block, in its first warp's lanes.  An FP64 addition holds a multiprocessor's pipe for 16 cycles a
// warp, so one warp adds the threads' sums, 12 additions (43 where every warp adds its own first).
__device__ __forceinline__ double block_sum64(double v, double *all)
{
    all[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
            v += all[w * 32 + threadIdx.x];
        v = warp_sum64(v);
    }
    return v;
}

// Sums of squares between these keep FP32's precision: none overflowed, and what
// underflowed is below 2^-33 of the sum.
constexpr float kSumLeast = 7.7e-34f, kSumMost = 1.2e30f;  // about 2^-110 and 2^100

// Runs of eight values that a thread has in flight: 64 bytes.
template <bool BF16>
constexpr int kAhead = BF16 ? 4 : 2;

// The sum of the squares of U runs, added to this thread's.
template <bool BF16, int U>
__device__ __forceinline__ void add_squares(const Values<BF16> (&v)[U], double &sum)
{
    F2 s2 = f2(0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < kVals / 2; ++i)
            s2 = f2_fma(v[u].pair(i), v[u].pair(i), s2);
    float a, b;
    f2_split(s2, a, b);
    const float s = a + b;
    if (s > kSumLeast && s < kSumMost) {
        sum += s;
        return;
    }
    uint32_t any = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < Values<BF16>::kWords; ++i)
            any |= v[u].r[i] & (BF16 ? 0x7FFF7FFFu : 0x7FFFFFFFu);
    if (any != 0)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < kVals / 2; ++i) {
                f2_split(v[u].pair(i), a, b);
                sum += static_cast<double>(a) * a + static_cast<double>(b) * b;
            }
}

// The squares of a block's part of a tensor.
template <bool BF16>
__device__ __forceinline__ void sum_part(const Tensor &t, const Part &p, double &sum)
{
    constexpr int E = BF16 ? 2 : 4, U = kAhead<BF16>;
    constexpr int kRun = kThreads * kVals * E;  // bytes from a thread's run to its next
    int64_t steps = (p.to - p.from) * kSteps;
    const int64_t first = p.from * kChunk + threadIdx.x * kVals;
    const char *from = static_cast<const char *>(t.src) + first * E;
    if ((t.flags & kGradSrcVector) && p.to * kChunk <= t.n) {
        for (; steps >= U; steps -= U, from += U * kRun) {
            Values<BF16> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                v[u].load(from + u * kRun);
            add_squares<BF16, U>(v, sum);
        }
        for (; steps > 0; --steps, from += kRun) {
            Values<BF16> v[1];
            v[0].load(from);
            add_squares<BF16, 1>(v, sum);
        }
        return;
    }
    for (int64_t left = t.n - first; steps > 0; --steps, from += kRun, left -= kThreads * kVals) {
        Values<BF16> v[1];
        if ((t.flags & kGradSrcVector) && left >= kVals)
            v[0].load(from);
        else
            v[0].load_some(from, left);
        add_squares<BF16, 1>(v, sum);
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    grad_norm_kernel(const __grid_constant__ Table<N> table, double *partial)
{
    __shared__ double part[kThreads];
    griddep_launch_dependents();
    griddep_wait();
    double sum = 0.0;
    Walk<N, false> walk(table);
    for (Part p; walk.next(p);) {
        const Tensor t(table.t[p.i]);
        if (t.flags & kGradSrcBf16)
            sum_part<true>(t, p, sum);
        else
            sum_part<false>(t, p, sum);
    }
    sum = block_sum64(sum, part);
    if (threadIdx.x == 0)
        partial[blockIdx.x] = sum;
}

// The sum of all squares from the blocks' sums.
__device__ __forceinline__ double total_of(const double *partial, int n, double *part)
{
    double s = static_cast<int>(threadIdx.x) < n ? __ldcg(partial + threadIdx.x) : 0.0;
    for (int i = threadIdx.x + kThreads; i < n; i += kThreads)
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
    __shared__ double part[kThreads];
    griddep_launch_dependents();
    griddep_wait();
    const double total = total_of(partial, n, part);
    if (threadIdx.x == 0)
        *norm = norm_of(total);
}

template <bool SRC>
__device__ __forceinline__ void scale(const Values<SRC> &v, F2 f, float (&o)[kVals])
{
#pragma unroll
    for (int i = 0; i < kVals / 2; ++i)
        f2_split(f2_mul(v.pair(i), f), o[2 * i], o[2 * i + 1]);
}

// A block's part of a tensor times the factor, from its end to its start.
template <bool SRC, bool DST>
__device__ __forceinline__ void clip_part(const Tensor &t, const Part &p, float factor)
{
    constexpr int ES = SRC ? 2 : 4, ED = DST ? 2 : 4, U = kAhead<SRC>;
    constexpr int64_t kRun = kThreads * kVals;
    const F2 f = f2(factor, factor);
    int64_t steps = (p.to - p.from) * kSteps;
    const int64_t last = p.to * kChunk - kRun + threadIdx.x * kVals;  // this thread's last run
    const char *from = static_cast<const char *>(t.src) + last * ES;
    char *to = static_cast<char *>(t.dst) + last * ED;
    constexpr uint32_t kBoth = kGradSrcVector | kGradDstVector;
    const bool vector = (t.flags & kBoth) == kBoth;
    if (vector && p.to * kChunk <= t.n) {
        for (; steps >= U; steps -= U, from -= U * kRun * ES, to -= U * kRun * ED) {
            Values<SRC> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                v[u].load(from - u * kRun * ES);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float o[kVals];
                scale(v[u], f, o);
                store_values<DST>(to - u * kRun * ED, o);
            }
        }
    }
    for (int64_t left = t.n - (last - (p.to - p.from) * kChunk + steps * kRun); steps > 0;
         --steps, from -= kRun * ES, to -= kRun * ED, left += kRun) {
        Values<SRC> v;
        if (vector && left >= kVals)
            v.load(from);
        else
            v.load_some(from, left);
        float o[kVals];
        scale(v, f, o);
        if (vector && left >= kVals)
            store_values<DST>(to, o);
        else
            store_some<DST>(to, left, o);
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    grad_clip_kernel(const __grid_constant__ Table<N> table, const double *partial, int n, float max_norm, float *norm)
{
    __shared__ double part[kThreads];
    __shared__ float block_factor;
    griddep_launch_dependents();
    Walk<N, true> walk(table);  // what does not depend on the norm comes before the wait for it
    Part p;
    bool any = walk.next(p);
    Tensor t(table.t[p.i]);
    griddep_wait();
    const double total = total_of(partial, n, part);
    if (threadIdx.x == 0) {
        block_factor = factor_of(total, max_norm);
        if (norm && blockIdx.x == 0)
            *norm = norm_of(total);
    }
    __syncthreads();
    const float factor = block_factor;
    while (any) {
        if (factor != 1.0f || t.src != t.dst) {  // what stays as it is need not be written
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
        any = walk.next(p);
        t = Tensor(table.t[p.i]);
    }
}

// One launch's table, and the number of its blocks.
template <int N>
unsigned fill_table(Table<N> &table, const GradTensor *tensors, int n, int num_sms)
{
    uint32_t chunks = 0;
    for (int i = 0; i < n; ++i) {
        table.t[i] = tensors[i];
        chunks += static_cast<uint32_t>(((tensors[i].n_flags >> kGradFlagBits) + kChunk - 1) / kChunk);
        table.end[i] = chunks;
    }
    table.chunks = chunks;
    const unsigned most = static_cast<unsigned>((num_sms < kGradSms ? num_sms : kGradSms) * kBlocksPerSm);
    // As many chunks to a block as the largest share is anyway, two at least where that still fills the multiprocessors: a
    // block's start and sum cost as much as those (4 M BF16 values 8 us with two chunks a block, 10 with four; 8 M 11.5
    // with 512 blocks of four, 12.2 with 608 of three or four).
    const unsigned share = std::max(2u, (chunks + most - 1) / most), sms = most / kBlocksPerSm;
    const unsigned blocks = std::max({1u, std::min(chunks, sms), (chunks + share - 1) / share});
    int i = 0;
    for (unsigned b = 0; b <= blocks; ++b) {
        const uint32_t chunk = static_cast<uint32_t>(static_cast<uint64_t>(chunks) * b / blocks);
        while (i + 1 < n && table.end[i] <= chunk)
            ++i;
        table.start[b] = static_cast<uint16_t>(i);
    }
    return blocks;
}

template <int N>
cudaError_t launch_tables(const GradTensor *tensors, int64_t n, bool clip, double *partial, float max_norm, float *norm,
                          int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    Table<N> table;
    int parts = 0;
    unsigned blocks = 0;
    for (int64_t at = 0; at < n; at += N) {
        blocks = fill_table(table, tensors + at, static_cast<int>(n - at < N ? n - at : N), num_sms);
        const cudaLaunchConfig_t cfg = row_launch(blocks, kThreads, 0, s, attr);
        const cudaError_t e = cudaLaunchKernelEx(&cfg, grad_norm_kernel<N>, table, partial + parts);
        if (e != cudaSuccess)
            return e;
        parts += static_cast<int>(blocks);
    }
    if (!clip) {
        const cudaLaunchConfig_t cfg = row_launch(1, kThreads, 0, s, attr);
        return cudaLaunchKernelEx(&cfg, grad_norm_finish_kernel, static_cast<const double *>(partial), parts, norm);
    }
    for (int64_t at = 0; at < n; at += N) {
        if (n > N)
            blocks = fill_table(table, tensors + at, static_cast<int>(n - at < N ? n - at : N), num_sms);
        const cudaLaunchConfig_t cfg = row_launch(blocks, kThreads, 0, s, attr);
        const cudaError_t e = cudaLaunchKernelEx(&cfg, grad_clip_kernel<N>, table, static_cast<const double *>(partial),
                                                 parts, max_norm, at == 0 ? norm : nullptr);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

// Few tensors take a short table: a launch copies its parameters (32 KB at most).
constexpr int kTables[5] = {32, 128, 320, 640, 1024};

int table_size(int64_t n)
{
    for (const int size : kTables)
        if (n <= size)
            return size;
    return kTables[4];
}

cudaError_t launch_any(const GradTensor *tensors, int64_t n, bool clip, double *partial, float max_norm, float *norm,
                       int num_sms, cudaStream_t s)
{
    switch (table_size(n)) {
    case kTables[0]:
        return launch_tables<kTables[0]>(tensors, n, clip, partial, max_norm, norm, num_sms, s);
    case kTables[1]:
        return launch_tables<kTables[1]>(tensors, n, clip, partial, max_norm, norm, num_sms, s);
    case kTables[2]:
        return launch_tables<kTables[2]>(tensors, n, clip, partial, max_norm, norm, num_sms, s);
    case kTables[3]:
        return launch_tables<kTables[3]>(tensors, n, clip, partial, max_norm, norm, num_sms, s);
    default:
        return launch_tables<kTables[4]>(tensors, n, clip, partial, max_norm, norm, num_sms, s);
    }
}

}  // namespace

size_t grad_workspace(int64_t n)
{
    const int64_t launches = (n + table_size(n) - 1) / table_size(n);
    return static_cast<size_t>(launches) * kMostBlocks * sizeof(double);
}

// Chunks of 4096 values of a launch are numbered in 32 bits.
bool grads_fit(const GradTensor *tensors, int64_t n)
{
    const int size = n > 0 ? table_size(n) : 1;
    int64_t chunks = 0;
    for (int64_t i = 0; i < n; ++i) {
        chunks = (i % size == 0 ? 0 : chunks) + ((tensors[i].n_flags >> kGradFlagBits) + kChunk - 1) / kChunk;
        if (chunks > 0x7FFFFFFF)
            return false;
    }
    return true;
}

cudaError_t launch_grad_norm(const GradTensor *tensors, int64_t n, double *partial, float *norm, int num_sms,
                             cudaStream_t s)
{
    return launch_any(tensors, n, false, partial, 0.0f, norm, num_sms, s);
}

cudaError_t launch_clip_grads(const GradTensor *tensors, int64_t n, double *partial, float max_norm, float *norm,
                              int num_sms, cudaStream_t s)
{
    return launch_any(tensors, n, n > 0, partial, max_norm, norm, num_sms, s);  // no tensors: the norm alone
}

}  // namespace mxg
