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
// A stable counting sort.  Every block owns a contiguous tile of slots and every
// warp of it a contiguous run.  (1) Each warp counts its run by expert in its own row
// of shared memory (lanes with the same expert find each other with match.any) and
// the columns are scanned over the warps.  (2) Each block learns the tiles' counts:
// over all tiles, which after a scan over the experts gives an expert's first row, and
// over the tiles before its own.  Up to eight tiles are one cluster and read each
// other's counts in distributed shared memory; more get them from a first kernel,
// beside which (1) runs.  (3) Each warp walks its run again and hands out rows in slot
// order.
//
// Latency-bound: 131072 slots are 2 MB of traffic.  What counts is that no SM gets
// many slots, since match.any and the scattered stores of the inverse map go
// through one SM slowly: 131072 slots of 64 experts take 7.6 us on 128 tiles, and took
// 28 us on one cluster.  A cluster saves a launch: 4000 slots 4.1 us against 4.6, 8198
// slots 4.5 against 4.7; at four steps a warp the counts' own kernel is faster (16000
// slots 6.2 us, 6.8 as a cluster), so clusters take up to three.
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortAhead = 4;
// A decode step's slots take a smaller block: 256 slots 2.5 us instead of 3.0.
constexpr int kFewThreads = 256;
constexpr int64_t kFewSlots = 4 * kFewThreads;
constexpr int kSortCluster = 8;
constexpr int64_t kClusterSlots = kSortCluster * 3 * kSortThreads;

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// *p in block `rank` of the cluster.
__device__ __forceinline__ int ld_cluster(const int *p, int rank)
{
    int v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
                 "ld.shared::cluster.b32 %0, [a];\n\t}"
                 : "=r"(v)
                 : "r"(smem_addr(p)), "r"(rank)
                 : "memory");
    return v;
}

template <typename ID>
__device__ __forceinline__ int expert_key(ID id, int groups)
{
    return id >= 0 && id < static_cast<ID>(groups) ? static_cast<int>(id) : groups;
}

// counts[tile][key]: the tile's slots of an expert (key `groups`: dropped).
template <typename ID>
__global__ void __launch_bounds__(kSortThreads)
    moe_count_kernel(const ID *ids, int64_t slots, int groups, int64_t tile, int *counts)
{
    __shared__ int total[kMaxSortGroups + 1];
    griddep_wait();
    // only now: the sort kernel reads the ids before it waits for this kernel, so what wrote them must be complete
    griddep_launch_dependents();
    const int tid = threadIdx.x, keys = groups + 1;
    for (int e = tid; e < keys; e += kSortThreads)
        total[e] = 0;
    __syncthreads();
    const int64_t s0 = blockIdx.x * tile, s1 = s0 + tile < slots ? s0 + tile : slots;
#pragma unroll 4
    for (int64_t s = s0 + tid; s < s1; s += kSortThreads)
        atomicAdd(&total[expert_key(ids[s], groups)], 1);  // counts only: the order does not matter
    __syncthreads();
    for (int e = tid; e < keys; e += kSortThreads)
        counts[static_cast<int64_t>(blockIdx.x) * keys + e] = total[e];
}

template <typename ID, int THREADS, bool CLUSTER>
__global__ void __launch_bounds__(THREADS)
    moe_sort_kernel(const ID *ids, int64_t slots, int groups, int64_t run, const int *counts, int64_t *offsets,
                    int32_t *row_of_slot, int32_t *slot_of_row)
{
    constexpr int kSortThreads = THREADS, kSortWarps = THREADS / 32;
    extern __shared__ int hist[];  // [kSortWarps][groups + 1]
    __shared__ int all[kMaxSortGroups + 1];    // slots of an expert (the last entry: dropped)
    __shared__ int own[CLUSTER ? kMaxSortGroups + 1 : 1];  // this tile's
    __shared__ int first[kMaxSortGroups + 1];  // slots of it in earlier tiles; then this tile's first row
    __shared__ int warp_part[kSortWarps];
    if (!counts)
        griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, keys = groups + 1;
    const int tile = static_cast<int>(blockIdx.x), tiles = static_cast<int>(gridDim.x);
    int *mine = hist + warp * keys;
    const int64_t s0 = (static_cast<int64_t>(tile) * kSortWarps + warp) * run;
    const int64_t s1 = s0 + run < slots ? s0 + run : slots;

    // four steps' ids are loaded together: one memory latency for 128 slots of a warp
    int key[kSortAhead];
    auto load_keys = [&](int64_t b) {
        ID id[kSortAhead];
#pragma unroll
        for (int i = 0; i < kSortAhead; ++i)
            id[i] = b + 32 * i + lane < s1 ? ids[b + 32 * i + lane] : 0;
#pragma unroll
        for (int i = 0; i < kSortAhead; ++i)
            key[i] = b + 32 * i + lane < s1 ? expert_key(id[i], groups) : -1;
    };
    load_keys(s0);
    for (int i = lane; i < keys; i += 32)
        mine[i] = 0;
    for (int e = tid; e < keys; e += kSortThreads)
        all[e] = first[e] = 0;
    __syncwarp();
    for (int64_t b = s0; b < s1; b += 32 * kSortAhead) {
        if (b > s0)
            load_keys(b);
#pragma unroll
        for (int i = 0; i < kSortAhead; ++i) {
            if (b + 32 * i >= s1)
                break;  // warp-uniform
            const uint32_t peers = __match_any_sync(0xFFFFFFFFu, key[i]);
            if (key[i] >= 0 && lane == __ffs(peers) - 1)
                mine[key[i]] += __popc(peers);
            __syncwarp();
        }
    }
    __syncthreads();
    // warps of this block that have a run
    const int64_t runs = (slots - static_cast<int64_t>(tile) * kSortWarps * run + run - 1) / run;
    const int busy = runs < kSortWarps ? static_cast<int>(runs > 0 ? runs : 0) : kSortWarps;
    for (int e = tid; e < keys; e += kSortThreads) {
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w)
            if (w < busy) {
                const int c = hist[w * keys + e];
                hist[w * keys + e] = sum;
                sum += c;
            }
        if (CLUSTER)
            own[e] = sum;
        else if (!counts)
            all[e] = sum;
    }
    if (CLUSTER) {
        cluster_barrier();
        for (int e = tid; e < keys; e += kSortThreads) {
            int sum = 0, before = 0;
#pragma unroll
            for (int r = 0; r < kSortCluster; ++r)
                if (r < tiles) {
                    const int n = ld_cluster(&own[e], r);
                    sum += n;
                    before += r < tile ? n : 0;
                }
            all[e] = sum;
            first[e] = before;
        }
    }
    if (counts) {
        griddep_wait();
        // a strip of tiles per group of `keys` threads; integer sums, so their order does not matter
        const int strips = kSortThreads > keys ? kSortThreads / keys : 1;
        for (int at = tid; at < strips * keys; at += kSortThreads) {
            const int strip = at / keys, e = at - strip * keys;
            int sum = 0, before = 0;
#pragma unroll 8
            for (int c = strip; c < tiles; c += strips) {
                const int n = counts[static_cast<int64_t>(c) * keys + e];
                sum += n;
                before += c < tile ? n : 0;
            }
            atomicAdd(&all[e], sum);
            atomicAdd(&first[e], before);
        }
    }
    griddep_launch_dependents();
    __syncthreads();
    // scan over the keys, consecutive ones to a thread
    constexpr int kKeys = kMaxSortGroups / THREADS + 1;
    const int e0 = kKeys * tid;
    int n[kKeys], mine_sum = 0;
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
        n[i] = e0 + i < keys ? all[e0 + i] : 0;
        mine_sum += n[i];
    }
    int incl = mine_sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        incl += lane >= o ? v : 0;
    }
    if (lane == 31)
        warp_part[warp] = incl;
    __syncthreads();
    if (e0 < keys) {
        int start = incl - mine_sum;
        for (int w = 0; w < warp; ++w)
            start += warp_part[w];
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            if (e0 + i < keys) {
                first[e0 + i] += start;
                if (tile == 0)
                    offsets[e0 + i] = start;  // the dropped slots' start is the last group's end
            }
            start += n[i];
        }
    }
    __syncthreads();
    for (int64_t b = s0; b < s1; b += 32 * kSortAhead) {
        if (run > 32 * kSortAhead)
            load_keys(b);
#pragma unroll
        for (int i = 0; i < kSortAhead; ++i) {
            if (b + 32 * i >= s1)
                break;  // warp-uniform
            const uint32_t peers = __match_any_sync(0xFFFFFFFFu, key[i]);
            const int at = key[i] >= 0 ? mine[key[i]] : 0;
            __syncwarp();
            if (key[i] >= 0) {
                if (lane == __ffs(peers) - 1)
                    mine[key[i]] = at + __popc(peers);
                const int64_t s = b + 32 * i + lane;
                const int row = first[key[i]] + at + __popc(peers & ((1u << lane) - 1u));
                row_of_slot[s] = key[i] < groups ? row : -1 - row;
                if (slot_of_row)
                    slot_of_row[row] = static_cast<int32_t>(s);
            }
            __syncwarp();
        }
    }
    if (CLUSTER)
        cluster_barrier();  // no block leaves while another may still read its counts
}

// ----------------------------------------------------------------- dispatch --
// A warp reads 512 or 1024 values of a token once, encodes them once and writes
// them to the rows of all the token's slots.  One unit of work per warp and a block
// for every four: with persistent warps, 32 an SM, the writes of 16384
// tokens x 2048 to 8 of 64 experts (346 MB) took 71 us, so they take 52 us (6.6
// TB/s).  Two chunks a warp keep more bytes in flight where there are warps enough
// (4099 x 4096, top 2, MXFP4: 10.0 us against 11.9); with few, one chunk is faster
// (32 x 2048, top 8: 1.8 us against 2.3).
//
// Blocks of dispatch and combine are four warps: a multiprocessor refills sooner than
// with eight (combine 41.7 us and 1.9 us at the sizes below; with eight 42.6 and 2.2).
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// Warps below which a call is latency-bound: sixteen a multiprocessor.
constexpr int64_t kFewWarps = 16;

// The row of a slot and whether it is dropped; an entry outside the table gives row -1.
__device__ __forceinline__ int slot_row(int r, int64_t slots, bool &dropped)
{
    dropped = r < 0;
    const int row = dropped ? -1 - r : r;
    return row < slots ? row : -1;
}

template <int IN, int FMT, int CHUNKS>
__global__ void __launch_bounds__(kThreads, 8) moe_dispatch_kernel(const DispatchParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int topk = static_cast<int>(p.topk);
    const uint32_t per_row = static_cast<uint32_t>((p.K + CHUNKS * kWarpVals - 1) / (CHUNKS * kWarpVals));
    const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5), token = unit / per_row;
    if (token >= p.tokens)
        return;
    const int64_t K = p.K, t = token, slots = p.tokens * topk;
    const int64_t k0 = static_cast<int64_t>(unit - token * per_row) * (CHUNKS * kWarpVals) + lane * kLaneVals;
    Raw16<IN> x[CHUNKS];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
        x[c].load(p.x + t * p.x_stride + (k0 + c * kWarpVals) * E, k0 + c * kWarpVals < K);
    const int32_t *entry = p.row_of_slot + t * topk;
    int r = lane < topk ? entry[lane] : 0;
    constexpr int kWords = FMT == kRowsBf16 ? 8 : FMT == kMxfp8 ? 4 : 2;
    uint32_t w[CHUNKS][kWords], scode[CHUNKS], word[CHUNKS];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        if constexpr (FMT == kRowsBf16) {  // a BF16 token is copied bit for bit
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[c][i] = IN == kBf16 ? x[c].r[0][i] : pack_bf16(x[c].at(2 * i), x[c].at(2 * i + 1));
        } else {
            float v[kLaneVals];
#pragma unroll
            for (int i = 0; i < kLaneVals; ++i)
                v[i] = x[c].at(i);
            const Codes16<FMT> q = mx_encode<FMT>(v, amax_bits(x[c]));
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[c][i] = q.w[i];
            scode[c] = q.scode;
            word[c] = tile_scale_word(q.scode, lane);
        }
    }
    for (int j = 0; j < topk; ++j) {
        if (j > 0 && (j & 31) == 0)
            r = j + lane < topk ? entry[j + lane] : 0;
        bool dropped;
        const int64_t row = slot_row(__shfl_sync(0xFFFFFFFFu, r, j & 31), slots, dropped);
        if (row < 0)
            continue;  // warp-uniform
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const int64_t k = k0 + c * kWarpVals;
            const bool inside = k < K;
            uint32_t o[kWords];
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                o[i] = dropped ? 0u : w[c][i];
            if constexpr (FMT == kRowsBf16) {
                if (inside)
                    st_row32(p.rows + (row * K + k) * 2, o);
            } else {
                if (inside && FMT == kMxfp8)
                    *reinterpret_cast<uint4 *>(p.rows + row * K + k) = make_uint4(o[0], o[1], o[2], o[kWords - 1]);
                if (inside && FMT == kMxfp4)
                    *reinterpret_cast<uint2 *>(p.rows + ((row * K + k) >> 1)) = make_uint2(o[0], o[1]);
                uint8_t *scales = p.scales + ((row * K + k) >> 5);
                if (p.mode == kScaleWords) {
                    if (inside && (lane & 7) == 0)
                        *reinterpret_cast<uint32_t *>(scales) = dropped ? 0x7F7F7F7Fu : word[c];
                } else if (inside && (lane & 1) == 0) {
                    *scales = static_cast<uint8_t>(dropped ? 127u : scode[c]);
                }
            }
        }
    }
}

// ------------------------------------------------------------------ combine --
// A warp sums 512 values of a token over its slots, in slot order; the rows of
// AHEAD slots are loaded before the first is added.  Neighbouring warps read
// neighbouring parts of the same rows.  Two slots ahead fit 64 registers, and 32 warps
// an SM then keep HBM busy: 8192 x 4096, top 2, with residual (269 MB) 41.7 us (6.4
// TB/s), 8192 x 2048, top 8 (336 MB) 50.7 us (6.6); four ahead on 24 warps 54.9.  With
// few warps the latency of a batch counts: 32 x 2048, top 8, takes 1.9 us eight ahead,
// 2.9 two ahead.
template <int IN, int AHEAD>
__global__ void __launch_bounds__(kThreads, AHEAD == 2 ? 8 : 3) moe_combine_kernel(const CombineParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, topk = static_cast<int>(p.topk);
    const uint32_t per_row = static_cast<uint32_t>((p.N + kWarpVals - 1) / kWarpVals);
    const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5), token = unit / per_row;
    if (token >= p.tokens)
        return;
    const int64_t t = token, slots = p.tokens * topk;
    const int64_t k = static_cast<int64_t>(unit - token * per_row) * kWarpVals + lane * kLaneVals;
    const bool inside = k < p.N;
    const int32_t *entry = p.row_of_slot + t * topk;
    const char *y0 = p.y + k * E;
    Raw16<IN> add;
    add.load(p.add + t * p.add_stride + k * E, inside && p.add != nullptr);
    float acc[kLaneVals];
    for (int j0 = 0; j0 < topk; j0 += AHEAD) {
        int r[AHEAD];
        float w[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            r[i] = j0 + i < topk ? entry[j0 + i] : -1;
            w[i] = p.weights && j0 + i < topk ? p.weights[t * topk + j0 + i] : 1.0f;
        }
        Raw16<IN> y[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const bool live = r[i] >= 0 && r[i] < slots;  // a dropped row is never read
            w[i] = live ? w[i] : 0.0f;
            y[i].load(y0 + r[i] * p.y_stride, inside && live);
        }
        if (j0 == 0) {
#pragma unroll
            for (int n = 0; n < kLaneVals; ++n)
                acc[n] = add.at(n);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int n = 0; n < kLaneVals; ++n)
                acc[n] = fmaf(w[i], y[i].at(n), acc[n]);
    }
    if (inside)
        store16<IN>(p.out + (t * p.N + k) * E, acc);
}

// A warp per slot: dy[row] = w * dout[t] and dw = <dout[t], y[row]>.  The next slot's
// entry is loaded ahead of its row.  More blocks than are resident even out the end: 32
// an SM 16384 x 512, top 8, 48 us, 3814 x 2048 FP32, top 8, 79 us; 16 an SM 48 and 86;
// without the entry ahead 52 and 85.
template <int IN>
__global__ void __launch_bounds__(kThreads) moe_combine_backward_kernel(const CombineBackParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t N = p.N, slots = p.tokens * p.topk;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    int64_t s = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    int next_entry = s < slots ? p.row_of_slot[s] : 0;
    float next_w = s < slots ? p.weights[s] : 0.0f;
    for (; s < slots; s += step) {
        const int64_t t = s / p.topk;
        bool dropped;
        const int64_t row = slot_row(next_entry, slots, dropped);
        const float w = dropped ? 0.0f : next_w;
        if (s + step < slots) {
            next_entry = p.row_of_slot[s + step];
            next_w = p.weights[s + step];
        }
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

unsigned strided_blocks(int64_t warps, int num_sms, int per_sm)
{
    const int64_t blocks = (warps + kWarps - 1) / kWarps, cap = static_cast<int64_t>(num_sms) * per_sm;
    return static_cast<unsigned>(blocks < cap ? blocks : cap);
}

unsigned warp_blocks(int64_t warps) { return static_cast<unsigned>((warps + kWarps - 1) / kWarps); }

template <int IN, int FMT>
cudaError_t launch_dispatch(const DispatchParams &p, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const int64_t units = p.tokens * ((p.K + kWarpVals - 1) / kWarpVals);
    if (units <= kFewWarps * num_sms) {
        const cudaLaunchConfig_t cfg = row_launch(warp_blocks(units), kThreads, 0, s, attr);
        return cudaLaunchKernelEx(&cfg, moe_dispatch_kernel<IN, FMT, 1>, p);
    }
    const int64_t pairs = p.tokens * ((p.K + 2 * kWarpVals - 1) / (2 * kWarpVals));
    const cudaLaunchConfig_t cfg = row_launch(warp_blocks(pairs), kThreads, 0, s, attr);
    return cudaLaunchKernelEx(&cfg, moe_dispatch_kernel<IN, FMT, 2>, p);
}

template <int IN>
cudaError_t launch_dispatch_fmt(const DispatchParams &p, int num_sms, cudaStream_t s)
{
    return p.fmt == kMxfp8   ? launch_dispatch<IN, kMxfp8>(p, num_sms, s)
           : p.fmt == kMxfp4 ? launch_dispatch<IN, kMxfp4>(p, num_sms, s)
                             : launch_dispatch<IN, kRowsBf16>(p, num_sms, s);
}

template <typename ID>
cudaError_t launch_sort(const ID *ids, int64_t slots, int groups, int64_t *offsets, int32_t *row_of_slot,
                        int32_t *slot_of_row, int *counts, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    if (slots <= kFewSlots) {
        constexpr int kFewWarps = kFewThreads / 32;
        const int64_t run = ((slots + kFewWarps - 1) / kFewWarps + 31) / 32 * 32;
        const size_t smem = static_cast<size_t>(kFewWarps) * (groups + 1) * sizeof(int);
        const cudaLaunchConfig_t cfg = row_launch(1, kFewThreads, smem, s, attr);
        return cudaLaunchKernelEx(&cfg, moe_sort_kernel<ID, kFewThreads, false>, ids, slots, groups, run,
                                  static_cast<const int *>(nullptr), offsets, row_of_slot, slot_of_row);
    }
    const int64_t tiles = sort_tiles(slots, groups), warps = tiles * kSortWarps;
    const int64_t run = ((slots + warps - 1) / warps + 31) / 32 * 32;
    if (slots <= kClusterSlots) {
        counts = nullptr;
    } else {
        const cudaLaunchConfig_t cfg = row_launch(static_cast<unsigned>(tiles), kSortThreads, 0, s, attr);
        const cudaError_t e =
            cudaLaunchKernelEx(&cfg, moe_count_kernel<ID>, ids, slots, groups, run * kSortWarps, counts);
        if (e != cudaSuccess)
            return e;
    }
    const size_t smem = static_cast<size_t>(kSortWarps) * (groups + 1) * sizeof(int);
    cudaLaunchConfig_t cfg = row_launch(static_cast<unsigned>(tiles), kSortThreads, smem, s, attr);
    if (counts || tiles == 1)
        return cudaLaunchKernelEx(&cfg, moe_sort_kernel<ID, kSortThreads, false>, ids, slots, groups, run,
                                  static_cast<const int *>(counts), offsets, row_of_slot, slot_of_row);
    cudaLaunchAttribute both[2] = {attr[0]};
    both[1].id = cudaLaunchAttributeClusterDimension;
    both[1].val.clusterDim.x = static_cast<unsigned>(tiles);
    both[1].val.clusterDim.y = 1;
    both[1].val.clusterDim.z = 1;
    cfg.attrs = both;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, moe_sort_kernel<ID, kSortThreads, true>, ids, slots, groups, run,
                              static_cast<const int *>(nullptr), offsets, row_of_slot, slot_of_row);
}

}  // namespace

// Tiles of a sort.  One block while its warps have at most four steps, then a
// cluster of up to eight with 1024 to 1536 slots each; past that 1024 slots a tile
// again, up to 128 tiles, and fewer where many experts make the tables of counts long
// (each tile reads them all).
int64_t sort_tiles(int64_t slots, int64_t groups)
{
    if (slots <= 4 * kSortThreads)
        return 1;
    const int64_t most = slots <= kClusterSlots ? kSortCluster : groups > 128 ? 64 : 128;
    const int64_t tiles = (slots + 1023) / 1024;
    return tiles < most ? tiles : most;
}

size_t sort_workspace(int64_t slots, int64_t groups)
{
    return slots <= kClusterSlots ? 0 : static_cast<size_t>(sort_tiles(slots, groups) * (groups + 1)) * sizeof(int);
}

cudaError_t launch_moe_sort(const void *ids, bool ids64, int64_t slots, int groups, int64_t *offsets,
                            int32_t *row_of_slot, int32_t *slot_of_row, int *counts, cudaStream_t s)
{
    return ids64 ? launch_sort(static_cast<const long long *>(ids), slots, groups, offsets, row_of_slot, slot_of_row,
                               counts, s)
                 : launch_sort(static_cast<const int *>(ids), slots, groups, offsets, row_of_slot, slot_of_row, counts,
                               s);
}

cudaError_t launch_moe_dispatch(const DispatchParams &p, int in_dtype, int num_sms, cudaStream_t s)
{
    return in_dtype == kBf16 ? launch_dispatch_fmt<kBf16>(p, num_sms, s) : launch_dispatch_fmt<kF32>(p, num_sms, s);
}

namespace {

template <int IN>
cudaError_t launch_combine(const CombineParams &p, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const int64_t units = p.tokens * ((p.N + kWarpVals - 1) / kWarpVals);
    const cudaLaunchConfig_t cfg = row_launch(warp_blocks(units), kThreads, 0, s, attr);
    return units <= kFewWarps * num_sms ? cudaLaunchKernelEx(&cfg, moe_combine_kernel<IN, 8>, p)
                                        : cudaLaunchKernelEx(&cfg, moe_combine_kernel<IN, 2>, p);
}

}  // namespace

cudaError_t launch_moe_combine(const CombineParams &p, int in_dtype, int num_sms, cudaStream_t s)
{
    return in_dtype == kBf16 ? launch_combine<kBf16>(p, num_sms, s) : launch_combine<kF32>(p, num_sms, s);
}

cudaError_t launch_moe_combine_backward(const CombineBackParams &p, int in_dtype, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = row_launch(strided_blocks(p.tokens * p.topk, num_sms, 32), kThreads, 0, s, attr);
    return in_dtype == kBf16 ? cudaLaunchKernelEx(&cfg, moe_combine_backward_kernel<kBf16>, p)
                             : cudaLaunchKernelEx(&cfg, moe_combine_backward_kernel<kF32>, p);
}

}  // namespace mxg
