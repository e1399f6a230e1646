// moe.cu -- mixture-of-experts routing around the grouped GEMM: token slots
// sorted by expert, token rows written to their experts' rows (quantised on the
// way), the experts' rows summed back with routing weights, and the gradients.
//
// A token t has topk slots s = t * topk + j.  The sort gives every slot a row
// (row_of_slot): the rows of expert 0 first, slots of one expert in slot order.
// A slot whose expert id is outside 0..groups-1 is dropped: its row lies past the
// last group's end and row_of_slot holds -1 - row.
#include "mx_block.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mxg {
namespace {

// --------------------------------------------------------------------- sort --
// A stable counting sort by one cluster.  Every warp owns a contiguous run of
// slots.  (1) Each warp counts its run by expert in its own row of shared memory
// (lanes with the same expert find each other with match.any); (2) columns are
// summed over the block's warps, over the cluster's blocks (distributed shared
// memory) and over the experts, which gives each (expert, block, warp) its first
// row; (3) each warp walks its run again and hands out rows in slot order.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCluster = 8;

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int ld_cluster(const int *p, int rank)
{
    uint32_t a;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

template <typename ID>
__global__ void __launch_bounds__(kSortThreads)
    moe_sort_kernel(const ID *ids, int64_t slots, int groups, int64_t run, int64_t *offsets, int32_t *row_of_slot,
                    int32_t *slot_of_row)
{
    extern __shared__ int hist[];  // [kSortWarps][groups + 1]
    __shared__ int total[kMaxSortGroups + 1];  // this block's slots of an expert (the last entry: dropped)
    __shared__ int first[kMaxSortGroups + 1];  // this block's first row of an expert
    __shared__ int warp_part[kSortWarps];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, keys = groups + 1;
    const int rank = static_cast<int>(blockIdx.x), blocks = static_cast<int>(gridDim.x);
    int *mine = hist + warp * keys;

    for (int i = lane; i < keys; i += 32)
        mine[i] = 0;
    __syncwarp();
    const int64_t s0 = (static_cast<int64_t>(rank) * kSortWarps + warp) * run;
    const int64_t s1 = s0 + run < slots ? s0 + run : slots;
    auto key_of = [&](int64_t s) -> int {
        if (s >= s1)
            return -1;
        const ID id = ids[s];
        return id >= 0 && id < static_cast<ID>(groups) ? static_cast<int>(id) : groups;
    };
    for (int64_t b = s0; b < s1; b += 32) {
        const int key = key_of(b + lane);
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, key);
        if (key >= 0 && lane == __ffs(peers) - 1)
            mine[key] += __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    for (int e = tid; e < keys; e += kSortThreads) {
        int sum = 0;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = hist[w * keys + e];
            hist[w * keys + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    cluster_barrier();
    // keys <= 513 < kSortThreads: one thread per expert
    int before = 0, all = 0;
    if (tid < keys)
        for (int r = 0; r < blocks; ++r) {
            const int c = ld_cluster(&total[tid], r);
            before += r < rank ? c : 0;
            all += c;
        }
    int incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        incl += lane >= o ? v : 0;
    }
    if (lane == 31)
        warp_part[warp] = incl;
    __syncthreads();
    int carry = 0;
    for (int w = 0; w < warp; ++w)
        carry += warp_part[w];
    const int start = carry + incl - all;
    if (tid < keys) {
        first[tid] = start + before;
        if (rank == 0)
            offsets[tid] = start;  // the dropped slots' start is the last group's end
    }
    __syncthreads();
    for (int64_t b = s0; b < s1; b += 32) {
        const int key = key_of(b + lane);
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, key);
        const int at = key >= 0 ? mine[key] : 0;
        __syncwarp();
        if (key >= 0) {
            if (lane == __ffs(peers) - 1)
                mine[key] = at + __popc(peers);
            const int row = first[key] + at + __popc(peers & ((1u << lane) - 1u));
            row_of_slot[b + lane] = key < groups ? row : -1 - row;
            if (slot_of_row)
                slot_of_row[row] = static_cast<int32_t>(b + lane);
        }
        __syncwarp();
    }
    cluster_barrier();  // no block leaves while another may still read its totals
}

// ----------------------------------------------------------------- dispatch --
// A warp reads 512 values of a token once, encodes them once and writes them to
// the rows of all the token's slots.
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The row of a slot and whether it is dropped; an entry outside the table gives row -1.
__device__ __forceinline__ int slot_row(int r, int64_t slots, bool &dropped)
{
    dropped = r < 0;
    const int row = dropped ? -1 - r : r;
    return row < slots ? row : -1;
}

template <int IN, int FMT>
__global__ void __launch_bounds__(kThreads) moe_dispatch_kernel(const DispatchParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t K = p.K, per_row = (K + kWarpVals - 1) / kWarpVals, units = p.tokens * per_row;
    const int64_t slots = p.tokens * p.topk;
    for (int64_t n = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); n < units;
         n += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t t = n / per_row, k0 = (n - t * per_row) * kWarpVals, k = k0 + lane * kLaneVals;
        const bool inside = k < K;
        Raw16<IN> x;
        x.load(p.x + t * p.x_stride + k * E, inside);
        int r = lane < p.topk ? p.row_of_slot[t * p.topk + lane] : 0;
        float v[kLaneVals];
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i)
            v[i] = x.at(i);
        Codes16<FMT == kMxfp4 ? kMxfp4 : kMxfp8> q, zero;
        if (FMT != kRowsBf16) {
            q = mx_encode<FMT == kMxfp4 ? kMxfp4 : kMxfp8>(v);
            zero = q;
#pragma unroll
            for (uint32_t &w : zero.w)
                w = 0;
            zero.scode = 127;
        }
        for (int64_t j = 0; j < p.topk; ++j) {
            if (j > 0 && (j & 31) == 0)
                r = j + lane < p.topk ? p.row_of_slot[t * p.topk + j + lane] : 0;
            bool dropped;
            const int64_t row = slot_row(__shfl_sync(0xFFFFFFFFu, r, static_cast<int>(j & 31)), slots, dropped);
            if (row < 0)
                continue;  // warp-uniform
            if (FMT == kRowsBf16) {
                uint32_t d[8];  // a BF16 token is copied bit for bit
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] = dropped ? 0u : IN == kBf16 ? x.r[0][i] : pack_bf16(v[2 * i], v[2 * i + 1]);
                if (inside)
                    st_row32(p.rows + (row * K + k) * 2, d);
            } else {
                const auto &o = dropped ? zero : q;
                if (inside)
                    store_codes(p.rows + row * (FMT == kMxfp8 ? K : K >> 1), k, o);
                store_scales(p.scales, p.mode, row, k0, K, lane, o.scode);
            }
        }
    }
}

// ------------------------------------------------------------------ combine --
// A warp sums 512 values of a token over its slots, in slot order.
template <int IN>
__global__ void __launch_bounds__(kThreads) moe_combine_kernel(const CombineParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t N = p.N, per_row = (N + kWarpVals - 1) / kWarpVals, units = p.tokens * per_row;
    const int64_t slots = p.tokens * p.topk;
    for (int64_t n = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); n < units;
         n += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t t = n / per_row, k = (n - t * per_row) * kWarpVals + lane * kLaneVals;
        const bool inside = k < N;
        float acc[kLaneVals];
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i)
            acc[i] = 0.0f;
        for (int64_t j = 0; j < p.topk; ++j) {
            bool dropped;
            const int64_t row = slot_row(p.row_of_slot[t * p.topk + j], slots, dropped);
            if (dropped || row < 0)
                continue;  // warp-uniform: a dropped row is never read
            const float w = p.weights ? p.weights[t * p.topk + j] : 1.0f;
            Raw16<IN> y;
            y.load(p.y + row * p.y_stride + k * E, inside);
#pragma unroll
            for (int i = 0; i < kLaneVals; ++i)
                acc[i] = fmaf(w, y.at(i), acc[i]);
        }
        if (p.add) {
            Raw16<IN> a;
            a.load(p.add + t * p.add_stride + k * E, inside);
#pragma unroll
            for (int i = 0; i < kLaneVals; ++i)
                acc[i] += a.at(i);
        }
        if (inside)
            store16<IN>(p.out + (t * N + k) * E, acc);
    }
}

// A warp per slot: dy[row] = w * dout[t] and dw = <dout[t], y[row]>.
template <int IN>
__global__ void __launch_bounds__(kThreads) moe_combine_backward_kernel(const CombineBackParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t N = p.N, slots = p.tokens * p.topk;
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); s < slots;
         s += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t t = s / p.topk;
        bool dropped;
        const int64_t row = slot_row(p.row_of_slot[s], slots, dropped);
        const float w = dropped ? 0.0f : p.weights[s];
        float dot = 0.0f;
        if (row >= 0) {
#pragma unroll 2
            for (int64_t k = lane * kLaneVals; k < N; k += kWarpVals) {
                Raw16<IN> d, y;
                d.load(p.dout + t * p.dout_stride + k * E, !dropped);
                y.load(p.y + row * p.y_stride + k * E, !dropped);
                float g[kLaneVals];
#pragma unroll
                for (int i = 0; i < kLaneVals; ++i) {
                    dot = fmaf(d.at(i), y.at(i), dot);
                    g[i] = w * d.at(i);
                }
                store16<IN>(p.dy + (row * N + k) * E, g);
            }
        }
        dot = warp_sum(dot);
        if (lane == 0)
            p.dweights[s] = dot;
    }
}

unsigned grid_for(int64_t warps, int num_sms)
{
    const int64_t blocks = (warps + kWarps - 1) / kWarps, cap = static_cast<int64_t>(num_sms) * 8;
    return static_cast<unsigned>(blocks < cap ? blocks : cap);
}

template <int IN>
cudaError_t launch_dispatch(const DispatchParams &p, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg =
        row_launch(grid_for(p.tokens * ((p.K + kWarpVals - 1) / kWarpVals), num_sms), kThreads, 0, s, attr);
    return p.fmt == kMxfp8   ? cudaLaunchKernelEx(&cfg, moe_dispatch_kernel<IN, kMxfp8>, p)
           : p.fmt == kMxfp4 ? cudaLaunchKernelEx(&cfg, moe_dispatch_kernel<IN, kMxfp4>, p)
                             : cudaLaunchKernelEx(&cfg, moe_dispatch_kernel<IN, kRowsBf16>, p);
}

}  // namespace

cudaError_t prepare_moe()
{
    const int most = kSortWarps * (kMaxSortGroups + 1) * static_cast<int>(sizeof(int));
    const cudaError_t e =
        cudaFuncSetAttribute(moe_sort_kernel<long long>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return e != cudaSuccess
               ? e
               : cudaFuncSetAttribute(moe_sort_kernel<int>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

cudaError_t launch_moe_sort(const void *ids, bool ids64, int64_t slots, int groups, int64_t *offsets,
                            int32_t *row_of_slot, int32_t *slot_of_row, cudaStream_t s)
{
    // a run of whole 32-slot steps per warp; one block while that gives each warp at most four steps
    const int blocks = slots <= 4 * kSortThreads ? 1 : kSortCluster;
    const int64_t warps = static_cast<int64_t>(blocks) * kSortWarps;
    const int64_t run = ((slots + warps - 1) / warps + 31) / 32 * 32;
    const size_t smem = static_cast<size_t>(kSortWarps) * (groups + 1) * sizeof(int);
    cudaLaunchAttribute attr[2];
    cudaLaunchAttribute one[1];
    cudaLaunchConfig_t cfg = row_launch(blocks, kSortThreads, smem, s, one);
    attr[0] = one[0];
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return ids64 ? cudaLaunchKernelEx(&cfg, moe_sort_kernel<long long>, static_cast<const long long *>(ids), slots,
                                      groups, run, offsets, row_of_slot, slot_of_row)
                 : cudaLaunchKernelEx(&cfg, moe_sort_kernel<int>, static_cast<const int *>(ids), slots, groups, run,
                                      offsets, row_of_slot, slot_of_row);
}

cudaError_t launch_moe_dispatch(const DispatchParams &p, int in_dtype, int num_sms, cudaStream_t s)
{
    return in_dtype == kBf16 ? launch_dispatch<kBf16>(p, num_sms, s) : launch_dispatch<kF32>(p, num_sms, s);
}

cudaError_t launch_moe_combine(const CombineParams &p, int in_dtype, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg =
        row_launch(grid_for(p.tokens * ((p.N + kWarpVals - 1) / kWarpVals), num_sms), kThreads, 0, s, attr);
    return in_dtype == kBf16 ? cudaLaunchKernelEx(&cfg, moe_combine_kernel<kBf16>, p)
                             : cudaLaunchKernelEx(&cfg, moe_combine_kernel<kF32>, p);
}

cudaError_t launch_moe_combine_backward(const CombineBackParams &p, int in_dtype, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = row_launch(grid_for(p.tokens * p.topk, num_sms), kThreads, 0, s, attr);
    return in_dtype == kBf16 ? cudaLaunchKernelEx(&cfg, moe_combine_backward_kernel<kBf16>, p)
                             : cudaLaunchKernelEx(&cfg, moe_combine_backward_kernel<kF32>, p);
}

}  // namespace mxg
