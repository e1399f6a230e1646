// embed.cu -- embedding rows of token ids, and the table's gradient.
//
//   out[t] = scale * table[ids[t]]                            (zeros for an id outside the table)
//   dtable[v] = add[v] + scale * sum over t with ids[t] = v of dy[t]
//
// The gradient is a sum of rows by key.  The ids are sorted (stable), so that the
// rows of an id are neighbours in token order; a warp sums 512 columns of 32 sorted
// (or 8) rows in FP32 registers and writes every run of an id that lies inside them at
// once.  Runs that cross into the next rows leave partial sums, which a last kernel adds in
// order.  No atomics on values: the same sums in every run.
#include "mx_block.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ int64_t load_id(const void *ids, bool wide, int64_t t)
{
    return wide ? static_cast<const int64_t *>(ids)[t] : static_cast<const int32_t *>(ids)[t];
}

// ------------------------------------------------------------------- lookup --
// A warp copies 512 values of a row, CHUNKS times: two where there are warps enough, so
// that more bytes are in flight behind one id (16384 x 8192 BF16 60.4 us, 6.3 TB/s of the
// rows written and the different rows read; bound by HBM), one for few tokens (8 x 8192:
// 1.8 us, an id's latency and a row's).
template <int IN, int OUT, int CHUNKS>
__global__ void __launch_bounds__(kThreads) embed_kernel(const EmbedParams p)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const uint32_t per_row = static_cast<uint32_t>((p.K + CHUNKS * kWarpVals - 1) / (CHUNKS * kWarpVals));
    const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5), token = unit / per_row;
    if (token >= p.tokens)
        return;
    const int64_t id = load_id(p.ids, p.ids64, token);
    const bool real = id >= 0 && id < p.vocab;
    const int64_t k0 = static_cast<int64_t>(unit - token * per_row) * (CHUNKS * kWarpVals) + lane * kLaneVals;
    Raw16<IN> x[CHUNKS];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
        x[c].load(p.table + id * p.table_stride + (k0 + c * kWarpVals) * E, real && k0 + c * kWarpVals < p.K);
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        float v[kLaneVals];
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i)
            v[i] = x[c].at(i) * p.scale;
        if (!real)  // zeros, whatever the sign of the scale
#pragma unroll
            for (int i = 0; i < kLaneVals; ++i)
                v[i] = 0.0f;
        const int64_t k = k0 + c * kWarpVals;
        if (k < p.K)
            store16<OUT>(p.out + (token * p.K + k) * ElemBytes<OUT>::value, v);
    }
}

// --------------------------------------------------------------------- sort --
// (id, token) in the order of the ids, tokens of one id in theirs.  Ids outside the
// table get the key `vocab`, the last one.
__device__ __forceinline__ uint32_t key_of(const void *ids, bool wide, int64_t t, uint32_t vocab)
{
    const int64_t id = load_id(ids, wide, t);
    return id >= 0 && id < vocab ? static_cast<uint32_t>(id) : vocab;
}

// Few tokens: every entry's place is the number of entries before it, counted by
// comparing it with all of them.  Id and token make one 32-bit number (the sizes below
// see to that), so a comparison is two instructions, and the blocks, of 64 entries each,
// have nothing to tell each other: no barrier between blocks (with the kernels that follow
// and find nothing to add, 1024 ids 5.1 us, by digits 10.3; 2048 7.2 and 10.8, 3000 12.4
// and 10.8, 8192 23.7 and 11.6).
constexpr int kRankThreads = 256;
constexpr int kRankEntries = 64;  // of a block: 16 lanes with four each
constexpr int kRankParts = kRankThreads / (kRankEntries / 4);
constexpr int kRankTokenBits = 11;
constexpr int64_t kRankTokens = 1 << kRankTokenBits;
constexpr int64_t kRankVocab = (1ll << (32 - kRankTokenBits)) - 1;

__global__ void __launch_bounds__(kRankThreads) embed_rank_kernel(const EmbedSortParams p)
{
    __shared__ __align__(16) uint32_t keys[kRankTokens];
    __shared__ int rank[kRankEntries];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, n = static_cast<int>(p.tokens), first = static_cast<int>(blockIdx.x) * kRankEntries;
    const int padded = (n + 4 * kRankParts - 1) / (4 * kRankParts) * (4 * kRankParts);
    if (tid < kRankEntries)
        rank[tid] = 0;
#pragma unroll 4
    for (int t = tid; t < padded; t += kRankThreads)  // what is past the end comes after everything
        keys[t] = t < n ? key_of(p.ids, p.ids64, t, p.vocab) << kRankTokenBits | static_cast<uint32_t>(t) : 0xFFFFFFFFu;
    __syncthreads();
    const int part = tid / (kRankEntries / 4), entry = tid % (kRankEntries / 4) * 4;
    uint32_t own[4];
    int before[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        own[i] = first + entry + i < n ? keys[first + entry + i] : 0u;
    const int steps = padded / (4 * kRankParts);
    const uint4 *from = reinterpret_cast<const uint4 *>(keys) + part * steps;
#pragma unroll 4
    for (int j = 0; j < steps; ++j) {
        const uint4 k = from[j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            before[i] += (k.x < own[i]) + (k.y < own[i]) + (k.z < own[i]) + (k.w < own[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        before[i] += __shfl_xor_sync(0xFFFFFFFFu, before[i], 16);  // the warp's other part
        if ((tid & 16) == 0)
            atomicAdd(&rank[entry + i], before[i]);  // whole numbers: the order does not matter
    }
    __syncthreads();
    if (tid < kRankEntries && first + tid < n) {
        const uint32_t k = keys[first + tid];
        p.entries0[rank[tid]] = make_uint2(k >> kRankTokenBits, k & (kRankTokens - 1));
    }
}

// More tokens: a stable radix sort in one cluster (32768 ids below 128256: 15 us, two
// passes of barriers, latencies and scattered stores).  Every block owns a contiguous part
// of the entries and every warp of it a contiguous run.  A pass counts its run's digits
// by warp, scans the counts over the warps, adds the other blocks' counts, and walks the
// run again to write the entries in order.  The blocks' counts pass through L2: from each
// other's shared memory the same 32 KB a block take 3000 cycles, here 1600.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortAhead = 4;
constexpr int kMaxDigits = 1 << kEmbedDigitBits;
constexpr int kHistStep = kSortWarps + 1;  // counts of a digit by warp, and a word between for the banks
static_assert(kSortWarps == 32 && kMaxDigits <= kSortThreads, "a lane for every warp, a thread for every digit");

__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(const EmbedSortParams p)
{
    extern __shared__ int hist[];  // [digits][kHistStep]
    __shared__ int first[kMaxDigits], warp_part[kSortWarps];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tile = static_cast<int>(blockIdx.x), tiles = static_cast<int>(gridDim.x);
    const int digits = 1 << p.bits;
    int *const mine = hist + warp;
    const int64_t s0 = (static_cast<int64_t>(tile) * kSortWarps + warp) * p.run;
    const int64_t s1 = s0 + p.run < p.tokens ? s0 + p.run : p.tokens;

    for (int pass = 0; pass < p.passes; ++pass) {
        const uint2 *from = pass & 1 ? p.entries0 : p.entries1;
        uint2 *to = pass & 1 ? p.entries1 : p.entries0;
        const int shift = pass * p.bits;
        uint2 e[kSortAhead];
        auto load = [&](int64_t b) {
#pragma unroll
            for (int i = 0; i < kSortAhead; ++i) {
                const int64_t s = b + 32 * i + lane;
                if (s >= s1)
                    e[i] = make_uint2(0xFFFFFFFFu, 0);
                else if (pass == 0)
                    e[i] = make_uint2(key_of(p.ids, p.ids64, s, p.vocab), static_cast<uint32_t>(s));
                else
                    e[i] = __ldcg(from + s);  // other blocks of the cluster wrote it
            }
        };
        auto digit = [&](const uint2 &v) { return static_cast<int>((v.x >> shift) & (digits - 1)); };
        load(s0);
        for (int i = tid; i < digits * kHistStep; i += kSortThreads)
            hist[i] = 0;
        __syncthreads();
        for (int64_t b = s0; b < s1; b += 32 * kSortAhead) {
            if (b > s0)
                load(b);
#pragma unroll
            for (int i = 0; i < kSortAhead; ++i) {
                if (b + 32 * i >= s1)
                    break;  // warp-uniform
                if (b + 32 * i + lane < s1)
                    atomicAdd(&mine[digit(e[i]) * kHistStep], 1);  // counts only: the order does not matter
            }
        }
        __syncthreads();
        // the counts of a digit scanned over the warps, half of them to a thread (a lane for every warp: 5500 cycles
        // instead of 1500, the shuffles)
        for (int t = tid; t - lane < 2 * digits; t += kSortThreads) {
            constexpr int kHalf = kSortWarps / 2;
            const bool live = t < 2 * digits;
            int *h = hist + (t >> 1) * kHistStep + (t & 1) * kHalf, n[kHalf], sum = 0;
#pragma unroll
            for (int i = 0; i < kHalf; ++i)
                sum += n[i] = live ? h[i] : 0;
            const int other = __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            if (live) {
                int at = t & 1 ? other : 0;
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    h[i] = at;
                    at += n[i];
                }
                if (t & 1)
                    __stcg(p.counts + tile * kMaxDigits + (t >> 1), at);
            }
        }
        cluster_sync();
        // one digit a thread: the digits' counts over all blocks, scanned, and those of the blocks before
        int total = 0, before = 0;
        if (tid < digits)
#pragma unroll
            for (int r = 0; r < kEmbedSortTiles; ++r)
                if (r < tiles) {
                    const int n = __ldcg(p.counts + r * kMaxDigits + tid);
                    total += n;
                    before += r < tile ? n : 0;
                }
        int incl = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            incl += lane >= o ? v : 0;
        }
        if (lane == 31)
            warp_part[warp] = incl;
        __syncthreads();
        int start = lane < warp ? warp_part[lane] : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            start += __shfl_xor_sync(0xFFFFFFFFu, start, o);
        if (tid < digits)
            first[tid] = start + incl - total + before;
        __syncthreads();
        for (int64_t b = s0; b < s1; b += 32 * kSortAhead) {
            if (p.run > 32 * kSortAhead)
                load(b);
#pragma unroll
            for (int i = 0; i < kSortAhead; ++i) {
                if (b + 32 * i >= s1)
                    break;  // warp-uniform
                const bool live = b + 32 * i + lane < s1;
                const int d = digit(e[i]);
                // the lanes with the same digit, a bit of it at a time (match.any takes its turns value by value)
                uint32_t peers = __ballot_sync(0xFFFFFFFFu, live);
                for (int bit = 0; bit < p.bits; ++bit) {
                    const uint32_t ones = __ballot_sync(0xFFFFFFFFu, (d >> bit) & 1);
                    peers &= (d >> bit) & 1 ? ones : ~ones;
                }
                const int at = live ? mine[d * kHistStep] : 0;
                __syncwarp();
                if (live) {
                    if (lane == __ffs(peers) - 1)
                        mine[d * kHistStep] = at + __popc(peers);
                    __stcg(to + first[d] + at + __popc(peers & ((1u << lane) - 1u)), e[i]);
                }
                __syncwarp();
            }
        }
        cluster_sync();  // entries are written, and no block reads counts any more
    }
}

// --------------------------------------------------------------------- sums --
// A warp takes 512 columns of RUN sorted rows, four of them in flight.  The rows that no
// token names are written by further blocks of the same launch: the sums are bound by
// latency, those by HBM (32768 x 4096 BF16 tokens into 128256 rows: 172 us together, 1.3
// GB at 7.6 TB/s with what stays in L2; the sums alone take 75).
// Sorted rows of a warp; fewer where few warps would each wait for 32 rows one after the other (1023 x 2048 FP32 added
// in place: 12 us, 20 with 32).
constexpr int kRun = 32, kShortRun = 8;
constexpr int64_t kShortRunWarps = 2048;

// Sixteen sums of a lane as the gradient's values at k of row `id`.
template <int OUT>
__device__ __forceinline__ void finish_row(const EmbedBackParams &p, uint32_t id, int64_t k, const float (&sum)[kLaneVals])
{
    constexpr int E = ElemBytes<OUT>::value;
    Raw16<OUT> add;
    add.load(p.add + (static_cast<int64_t>(id) * p.K + k) * E, p.add != nullptr);
    float v[kLaneVals];
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i)
        v[i] = fmaf(sum[i], p.scale, add.at(i));
    store16<OUT>(p.dtable + (static_cast<int64_t>(id) * p.K + k) * E, v);
}

// First entry whose id is not below `id`, found by the warp's 32 probes at a time.
__device__ __forceinline__ int64_t lower_bound(const EmbedBackParams &p, uint32_t id, int64_t from)
{
    const int lane = threadIdx.x & 31;
    int64_t n = p.tokens - from;
    while (n > 0) {
        const int64_t step = (n + 31) / 32, at = lane * step;
        const uint32_t below = __popc(__ballot_sync(0xFFFFFFFFu, at < n && p.entries[from + at].x < id));
        if (below == 0)
            break;
        // the last probe below `id` and what follows it up to the next probe
        const int64_t skip = (below - 1) * step + 1, end = below * step < n ? below * step : n;
        from += skip;
        n = end - skip;
    }
    return from;
}

// Row v as it is without the tokens.
template <int OUT>
__device__ __forceinline__ void fill_row(const EmbedBackParams &p, int64_t v)
{
    constexpr int E = ElemBytes<OUT>::value;
    for (int64_t k = (threadIdx.x & 31) * kLaneVals; k < p.K; k += kWarpVals) {
        Raw16<OUT> a;
        a.load(p.add + (v * p.K + k) * E, p.add != nullptr);
#pragma unroll
        for (int l = 0; l < Raw16<OUT>::kParts; ++l)
            st_row32(p.dtable + (v * p.K + k) * E + 32 * l, a.r[l]);
    }
}

// The warp writes those of the rows v0 .. v0 + rows - 1 whose id does not occur.
template <int OUT>
__device__ __forceinline__ void fill_rows(const EmbedBackParams &p, int64_t v0, int64_t rows)
{
    const int lane = threadIdx.x & 31;
    const int64_t v1 = v0 + rows < p.vocab ? v0 + rows : p.vocab;
    if (v0 >= v1)
        return;
    int64_t at = lower_bound(p, static_cast<uint32_t>(v0), 0);
    for (int64_t v = v0; v < v1;) {
        const uint32_t id = at + lane < p.tokens ? p.entries[at + lane].x : p.vocab;
        const uint32_t next = __shfl_sync(0xFFFFFFFFu, id, 0);  // the next id that occurs
        for (const int64_t end = next < v1 ? next : v1; v < end; ++v)
            fill_row<OUT>(p, v);
        ++v;  // past the id that occurs
        const int same = __popc(__ballot_sync(0xFFFFFFFFu, id == next));
        at = same < 32 ? at + same : lower_bound(p, next + 1, at + 32);
    }
}

// The first `sum_blocks` blocks sum, RUN sorted rows a warp; the others write the rows
// whose id does not occur, `rows` to a warp.
template <int IN, int OUT, int RUN>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const EmbedBackParams p, uint32_t sum_blocks, int64_t rows)
{
    constexpr int E = ElemBytes<IN>::value;
    constexpr int kAhead = IN == kBf16 || RUN == kShortRun ? 4 : 2;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t K = p.K;
    if (blockIdx.x >= sum_blocks) {
        const int64_t warp = static_cast<int64_t>(blockIdx.x - sum_blocks) * kWarps + (threadIdx.x >> 5);
        fill_rows<OUT>(p, warp * rows, rows);
        return;
    }
    const uint32_t slices = static_cast<uint32_t>((K + kWarpVals - 1) / kWarpVals);
    const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5), run = unit / slices;
    const int64_t c0 = static_cast<int64_t>(run) * RUN, k = (unit - run * slices) * kWarpVals + lane * kLaneVals;
    if (c0 >= p.tokens)
        return;
    const bool inside = k < K;
    const uint2 none = make_uint2(p.vocab, 0);
    const uint2 e = lane < RUN && c0 + lane < p.tokens ? p.entries[c0 + lane] : none;
    const uint32_t before = c0 > 0 ? p.entries[c0 - 1].x : 0xFFFFFFFFu;
    const uint32_t after = c0 + RUN < p.tokens ? p.entries[c0 + RUN].x : 0xFFFFFFFFu;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, e.x < p.vocab));  // ids outside the table come last
    bool open = __shfl_sync(0xFFFFFFFFu, e.x, 0) == before;           // the current run began before these rows
    float sum[kLaneVals];
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i)
        sum[i] = 0.0f;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        Raw16<IN> x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t t = __shfl_sync(0xFFFFFFFFu, e.y, (i0 + j) & 31);
            x[j].load(p.dy + t * p.dy_stride + k * E, inside && i0 + j < n);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j;
            if (i >= n)
                break;  // warp-uniform
#pragma unroll
            for (int l = 0; l < kLaneVals; ++l)
                sum[l] += x[j].at(l);
            const uint32_t id = __shfl_sync(0xFFFFFFFFu, e.x, i);
            const uint32_t next = i == RUN - 1 ? after : __shfl_sync(0xFFFFFFFFu, e.x, (i + 1) & 31);
            if (i < RUN - 1 && next == id)
                continue;
            const bool goes_on = next == id;
            if (inside) {
                if (open || goes_on) {
                    char *part = reinterpret_cast<char *>(p.partial + (static_cast<int64_t>(run) * 2 + (open ? 0 : 1)) * K + k);
                    store16<kF32>(part, sum);
                } else {
                    finish_row<OUT>(p, id, k, sum);
                }
            }
            open = false;
#pragma unroll
            for (int l = 0; l < kLaneVals; ++l)
                sum[l] = 0.0f;
        }
    }
}

// Runs over more than one warp's rows: a warp looks at the run that leaves RUN rows
// and began in them, and adds its partial sums in order (11 us for 1024 runs of 4096
// columns: three latencies and the barrier of the long ones).  Long ones (more than kLong
// parts) are added by all warps of the block, each every kJoinWarps-th part.
constexpr int kJoinWarps = 8;
constexpr int kLong = 8;

template <int OUT, int RUN>
__global__ void __launch_bounds__(32 * kJoinWarps) embed_join_kernel(const EmbedBackParams p)
{
    __shared__ float sums[kJoinWarps][kWarpVals];
    __shared__ int parts_of[kJoinWarps];
    __shared__ uint32_t id_of[kJoinWarps];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t K = p.K, k = static_cast<int64_t>(blockIdx.y) * kWarpVals + lane * kLaneVals;
    const bool inside = k < K;
    const int64_t run0 = static_cast<int64_t>(blockIdx.x) * kJoinWarps;
    auto add_part = [&](float (&sum)[kLaneVals], int64_t run, int j) {  // the j-th part of a run that began in `run`
        const char *part = reinterpret_cast<const char *>(p.partial + ((run + j) * 2 + (j == 0 ? 1 : 0)) * K + k);
        Raw16<kF32> x;
        x.load(part, inside);
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i)
            sum[i] += x.at(i);
    };
    float sum[kLaneVals];
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i)
        sum[i] = 0.0f;
    {
        const int64_t run = run0 + warp, c0 = run * RUN, end = c0 + RUN;
        int parts = 0;
        uint32_t id = p.vocab;
        if (end < p.tokens) {
            id = p.entries[end - 1].x;
            const bool here = c0 == 0 || p.entries[c0 - 1].x != id;  // where the last id began
            if (id < p.vocab && here && p.entries[end].x == id) {
                parts = 1;
                for (int64_t c = end + static_cast<int64_t>(lane) * RUN;; c += 32 * RUN) {
                    const uint32_t same = __ballot_sync(0xFFFFFFFFu, c < p.tokens && p.entries[c].x == id);
                    parts += __popc(same);  // ids are sorted: a prefix of the lanes
                    if (same != 0xFFFFFFFFu)
                        break;
                }
            }
        }
        if (lane == 0) {
            parts_of[warp] = parts;
            id_of[warp] = id;
        }
        if (parts > 0 && parts <= kLong) {
#pragma unroll 2
            for (int j = 0; j < parts; ++j)
                add_part(sum, run, j);
            if (inside)
                finish_row<OUT>(p, id, k, sum);
        }
    }
    __syncthreads();
    for (int w = 0; w < kJoinWarps; ++w) {
        const int parts = parts_of[w];
        if (parts <= kLong)
            continue;  // block-uniform
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i)
            sum[i] = 0.0f;
#pragma unroll 4
        for (int j = warp; j < parts; j += kJoinWarps)
            add_part(sum, run0 + w, j);
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i)
            sums[warp][i * 32 + lane] = sum[i];
        __syncthreads();
        if (warp == 0) {
            for (int o = 1; o < kJoinWarps; ++o)
#pragma unroll
                for (int i = 0; i < kLaneVals; ++i)
                    sum[i] += sums[o][i * 32 + lane];
            if (inside)
                finish_row<OUT>(p, id_of[w], k, sum);
        }
        __syncthreads();
    }
}

// A handful of tokens: no sort.  Every warp reads all ids, two a lane; the warp of an id's
// first token adds its rows, in token order, and the others of that id nothing.  One
// launch instead of three: the host's part of a call is 3.5 us instead of 8.
constexpr int64_t kFewTokens = 64;

template <int IN, int OUT>
__global__ void __launch_bounds__(kThreads)
    embed_few_kernel(const EmbedBackParams p, const void *ids, bool ids64, uint32_t sum_blocks, int64_t rows)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t K = p.K;
    uint32_t id[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        id[i] = lane + 32 * i < p.tokens ? key_of(ids, ids64, lane + 32 * i, p.vocab) : p.vocab;
    if (blockIdx.x >= sum_blocks) {  // `rows`, 32 at most, to a warp: a bit for every one that occurs
        const int64_t v0 = (static_cast<int64_t>(blockIdx.x - sum_blocks) * kWarps + warp) * rows;
        uint32_t occurs = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (id[i] >= v0 && id[i] < v0 + rows)
                occurs |= 1u << (id[i] - v0);
        occurs = __reduce_or_sync(0xFFFFFFFFu, occurs);
        for (int64_t v = v0; v < v0 + rows && v < p.vocab; ++v)
            if (!((occurs >> (v - v0)) & 1))
                fill_row<OUT>(p, v);
        return;
    }
    const uint32_t slices = static_cast<uint32_t>((K + kWarpVals - 1) / kWarpVals);
    const uint32_t unit = blockIdx.x * kWarps + warp, token = unit / slices;
    if (token >= p.tokens)
        return;
    const int64_t k = (unit - token * slices) * kWarpVals + lane * kLaneVals;
    const uint32_t lo = __shfl_sync(0xFFFFFFFFu, id[0], token & 31), hi = __shfl_sync(0xFFFFFFFFu, id[1], token & 31);
    const uint32_t mine = token < 32 ? lo : hi;
    unsigned long long same = __ballot_sync(0xFFFFFFFFu, id[0] == mine) |
                              static_cast<unsigned long long>(__ballot_sync(0xFFFFFFFFu, id[1] == mine)) << 32;
    if (mine >= p.vocab || __ffsll(same) - 1 != static_cast<int>(token) || k >= K)
        return;
    float sum[kLaneVals];
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i)
        sum[i] = 0.0f;
    while (same) {
        Raw16<IN> x[4];
        int n = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t t = __ffsll(same) - 1;
            x[j].load(p.dy + t * p.dy_stride + k * E, same != 0);
            n += same != 0;
            same &= same - 1;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < n)
#pragma unroll
                for (int i = 0; i < kLaneVals; ++i)
                    sum[i] += x[j].at(i);
    }
    finish_row<OUT>(p, mine, k, sum);
}

unsigned warp_blocks(int64_t warps) { return static_cast<unsigned>((warps + kWarps - 1) / kWarps); }

template <int IN, int OUT>
cudaError_t launch_lookup(const EmbedParams &p, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const int64_t units = p.tokens * ((p.K + kWarpVals - 1) / kWarpVals);
    if (units <= 16ll * num_sms) {
        const cudaLaunchConfig_t cfg = row_launch(warp_blocks(units), kThreads, 0, s, attr);
        return cudaLaunchKernelEx(&cfg, embed_kernel<IN, OUT, 1>, p);
    }
    const int64_t pairs = p.tokens * ((p.K + 2 * kWarpVals - 1) / (2 * kWarpVals));
    const cudaLaunchConfig_t cfg = row_launch(warp_blocks(pairs), kThreads, 0, s, attr);
    return cudaLaunchKernelEx(&cfg, embed_kernel<IN, OUT, 2>, p);
}

int key_bits(int64_t vocab)
{
    int bits = 1;
    while ((vocab >> bits) != 0)  // the keys are 0 .. vocab
        ++bits;
    return bits;
}

cudaError_t launch_sort(const EmbedSortParams &p, int tiles, cudaStream_t s)
{
    cudaLaunchAttribute attr[1], both[2];
    if (p.passes == 0) {
        const cudaLaunchConfig_t cfg =
            row_launch(static_cast<unsigned>((p.tokens + kRankEntries - 1) / kRankEntries), kRankThreads, 0, s, attr);
        return cudaLaunchKernelEx(&cfg, embed_rank_kernel, p);
    }
    const size_t smem = static_cast<size_t>(kHistStep) * sizeof(int) << p.bits;
    cudaLaunchConfig_t cfg = row_launch(static_cast<unsigned>(tiles), kSortThreads, smem, s, attr);
    both[0] = attr[0];
    both[1].id = cudaLaunchAttributeClusterDimension;
    both[1].val.clusterDim.x = static_cast<unsigned>(tiles);
    both[1].val.clusterDim.y = 1;
    both[1].val.clusterDim.z = 1;
    cfg.attrs = both;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, embed_sort_kernel, p);
}

template <int IN, int OUT, int RUN>
cudaError_t launch_runs(const EmbedBackParams &p, bool fill, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const int64_t slices = (p.K + kWarpVals - 1) / kWarpVals, runs = (p.tokens + RUN - 1) / RUN;
    const unsigned sum_blocks = warp_blocks(runs * slices);
    const int64_t row = p.K * ElemBytes<OUT>::value, rows = row >= 16384 ? 1 : 16384 / row;  // of a warp that fills
    const unsigned fill_blocks = fill ? warp_blocks((p.vocab + rows - 1) / rows) : 0;
    cudaLaunchConfig_t cfg = row_launch(sum_blocks + fill_blocks, kThreads, 0, s, attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, embed_sum_kernel<IN, OUT, RUN>, p, sum_blocks, rows);
    if (e != cudaSuccess || runs == 1)
        return e;
    cfg = row_launch(static_cast<unsigned>((runs + kJoinWarps - 1) / kJoinWarps), 32 * kJoinWarps, 0, s, attr);
    cfg.gridDim.y = static_cast<unsigned>(slices);
    return cudaLaunchKernelEx(&cfg, embed_join_kernel<OUT, RUN>, p);
}

bool short_runs(int64_t tokens, int64_t K)
{
    return tokens / kRun * ((K + kWarpVals - 1) / kWarpVals) < kShortRunWarps;
}

template <int IN, int OUT>
cudaError_t launch_few(const EmbedBackParams &p, const void *ids, bool ids64, bool fill, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const unsigned sum_blocks = warp_blocks(p.tokens * ((p.K + kWarpVals - 1) / kWarpVals));
    const int64_t row = p.K * ElemBytes<OUT>::value, wanted = row >= 16384 ? 1 : 16384 / row, rows = wanted < 32 ? wanted : 32;
    const unsigned fill_blocks = fill ? warp_blocks((p.vocab + rows - 1) / rows) : 0;
    const cudaLaunchConfig_t cfg = row_launch(sum_blocks + fill_blocks, kThreads, 0, s, attr);
    return cudaLaunchKernelEx(&cfg, embed_few_kernel<IN, OUT>, p, ids, ids64, sum_blocks, rows);
}

template <int IN, int OUT>
cudaError_t launch_sums(const EmbedBackParams &p, bool fill, cudaStream_t s)
{
    return short_runs(p.tokens, p.K) ? launch_runs<IN, OUT, kShortRun>(p, fill, s)
                                     : launch_runs<IN, OUT, kRun>(p, fill, s);
}

int64_t round_up(int64_t n) { return (n + 31) / 32 * 32; }

}  // namespace

cudaError_t prepare_embed()
{
    const cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kHistStep * kMaxDigits * static_cast<int>(sizeof(int)));
    return e == cudaSuccess ? cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)
                            : e;
}

cudaError_t launch_embed(const EmbedParams &p, int in_dtype, int out_dtype, int num_sms, cudaStream_t s)
{
    if (in_dtype == kBf16)
        return out_dtype == kBf16 ? launch_lookup<kBf16, kBf16>(p, num_sms, s) : launch_lookup<kBf16, kF32>(p, num_sms, s);
    return out_dtype == kBf16 ? launch_lookup<kF32, kBf16>(p, num_sms, s) : launch_lookup<kF32, kF32>(p, num_sms, s);
}

// Blocks of the sort.
int sort_tiles(int64_t tokens)
{
    int tiles = 1;
    while (tiles < kEmbedSortTiles && static_cast<int64_t>(tiles) * kSortThreads < tokens)
        tiles *= 2;
    return tiles;
}

// Two buffers of entries, and two rows of partial sums for every run, where the sort has its counts before.
EmbedWorkspace embed_workspace(int64_t tokens, int64_t K)
{
    EmbedWorkspace w = {};
    if (tokens <= kFewTokens)
        return w;
    w.entries[0] = 0;
    w.entries[1] = round_up(tokens * static_cast<int64_t>(sizeof(uint2)));
    w.partial = 2 * w.entries[1];
    const int64_t run = short_runs(tokens, K) ? kShortRun : kRun, runs = (tokens + run - 1) / run;
    const int64_t sums = runs > 1 ? runs * 2 * K * 4 : 0, counts = sort_tiles(tokens) * kMaxDigits * 4;
    w.bytes = static_cast<size_t>(w.partial + (sums > counts ? sums : counts));
    return w;
}

cudaError_t launch_embed_backward(EmbedBackParams p, const void *ids, bool ids64, char *workspace, int in_dtype,
                                  int out_dtype, cudaStream_t s)
{
    const bool fill = p.add != p.dtable;  // where the gradient is added in place, no other row is touched
    if (p.tokens <= kFewTokens) {
        if (in_dtype == kBf16)
            return out_dtype == kBf16 ? launch_few<kBf16, kBf16>(p, ids, ids64, fill, s)
                                      : launch_few<kBf16, kF32>(p, ids, ids64, fill, s);
        return out_dtype == kBf16 ? launch_few<kF32, kBf16>(p, ids, ids64, fill, s)
                                  : launch_few<kF32, kF32>(p, ids, ids64, fill, s);
    }
    const EmbedWorkspace w = embed_workspace(p.tokens, p.K);
    EmbedSortParams o;
    o.ids = ids;
    o.ids64 = ids64;
    o.tokens = p.tokens;
    o.vocab = p.vocab;
    const int bits = key_bits(p.vocab);
    // 0: by counting
    o.passes = p.tokens <= kRankTokens && p.vocab < kRankVocab ? 0 : (bits + kEmbedDigitBits - 1) / kEmbedDigitBits;
    o.bits = o.passes > 0 ? (bits + o.passes - 1) / o.passes : 0;
    const int tiles = sort_tiles(p.tokens);
    const int64_t warps = static_cast<int64_t>(tiles) * kSortWarps;
    o.run = ((p.tokens + warps - 1) / warps + 31) / 32 * 32;
    o.entries0 = reinterpret_cast<uint2 *>(workspace + w.entries[0]);
    o.entries1 = reinterpret_cast<uint2 *>(workspace + w.entries[1]);
    o.counts = reinterpret_cast<int *>(workspace + w.partial);
    const cudaError_t e = launch_sort(o, tiles, s);
    if (e != cudaSuccess)
        return e;
    p.entries = o.passes > 0 && o.passes % 2 == 0 ? o.entries1 : o.entries0;
    p.partial = reinterpret_cast<float *>(workspace + w.partial);
    if (in_dtype == kBf16)
        return out_dtype == kBf16 ? launch_sums<kBf16, kBf16>(p, fill, s) : launch_sums<kBf16, kF32>(p, fill, s);
    return out_dtype == kBf16 ? launch_sums<kF32, kBf16>(p, fill, s) : launch_sums<kF32, kF32>(p, fill, s);
}

}  // namespace mxg
