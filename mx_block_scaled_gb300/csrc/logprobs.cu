// logprobs.cu -- log probabilities of given tokens with the distribution's entropy
// and its most probable tokens, and the logits' gradient.
//
//   z_v = scale * (x_v - max x);  S = sum exp(z_v)
//   logprob = z_target - ln S;  entropy = ln S - sum exp(z_v) z_v / S
//   dx_v = scale * (dlogprob * ([v = target] - p_v) - dentropy * p_v * (ln p_v + entropy))
//
// One pass over a row: every thread sums 2^(c (x - r)), c = scale * log2(e), and its
// product with the exponent relative to a reference r of its own, which it moves only
// where a value is more than 2^kMargin above it; the sums are rebased to the row's
// maximum at the end.  The most probable tokens: the threads' own maxima give a value
// that at least `top` logits reach; the few logits that reach it are collected from
// the chunks whose maximum does, and ranked against each other.
//
// Bound by HBM for long rows: 4096 x 128256 BF16 153 us (6.9 TB/s), with entropy 157 (a
// value costs one 2^t and eight packed or paired instructions), with the 20 most
// probable 172, with both 183 (a row's last steps, 3 us, are covered by the three other
// blocks of its multiprocessor); 16 such rows on clusters of eight blocks, from L2, 3.7, 4.1,
// 6.7 and 7.0 us (the last from HBM 7.8), latency: two memory accesses, two cluster barriers,
// with the most probable ones four and three.
#include <algorithm>
#include <cfloat>
#include <cstdint>

#include "mx_block.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kThreads = 256;  // of a block at most
constexpr int kWarps = kThreads / 32;
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMargin = 3.0f;
constexpr int kFetchAhead = 32768;  // bytes of a later row
constexpr int kCandidates = 512, kGroupList = 384;
constexpr int kKeptMaxima = 32;  // maxima that a thread keeps, of one or more chunks each; a bit of a word for every one

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Below this a logit's share of the sums is zero, relative to the reference r: its
// exponent is -1000 or less.  Values are raised to it so that an infinite one gives 0
// times a finite number.  At least a BF16 step below r; -inf where there is no such
// number, or its exponent times `factor` is not finite (the sums then guard every product).
__device__ __forceinline__ float floor_of(float r, float c, float factor = 1.0f)
{
    const float f = fminf(r - 1000.0f / c, r - fabsf(r) * 0.0078125f), low = __bfloat162float(__float2bfloat16_rd(f));
    return (r - low) * c * factor <= FLT_MAX ? low : neg_inf();
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// 32 bytes of a row: sixteen BF16 or eight FP32 values.
template <int DT>
struct Chunk {
    static constexpr int kVals = 32 / ElemBytes<DT>::value;
    uint32_t r[8];

    __device__ __forceinline__ void load(const char *p) { ld_row32(p, r); }
    __device__ __forceinline__ float at(int i) const
    {
        if constexpr (DT == kBf16)
            return __uint_as_float((i & 1) ? (r[i >> 1] & 0xFFFF0000u) : (r[i >> 1] << 16));
        else
            return __uint_as_float(r[i]);
    }
    __device__ __forceinline__ F2 pair(int i) const
    {
        if constexpr (DT == kBf16)
            return f2_bf16(r[i]);
        else
            return f2(at(2 * i), at(2 * i + 1));
    }
    // the largest value; NaN if one is
    __device__ __forceinline__ float max() const
    {
        if constexpr (DT == kBf16) {
            uint32_t m = r[0];
#pragma unroll
            for (int i = 1; i < 8; ++i)
                asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(r[i]));
            return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
        } else {
            float m = at(0);
#pragma unroll
            for (int i = 1; i < 7; i += 2)
                asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(at(i)), "f"(at(i + 1)));
            return max_nan(m, at(7));
        }
    }
    // the values, raised to `low`
    __device__ __forceinline__ Chunk raised(float low) const
    {
        Chunk y;
        const uint32_t l = DT == kBf16 ? pack_bf16(low, low) : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (DT == kBf16)
                asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y.r[i]) : "r"(r[i]), "r"(l));
            else
                y.r[i] = __float_as_uint(max_nan(at(i), low));
        }
        return y;
    }
};

template <int DT>
__device__ __forceinline__ float load_one(const char *p)
{
    if constexpr (DT == kBf16)
        return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(p)) << 16);
    else
        return *reinterpret_cast<const float *>(p);
}

template <int DT>
__device__ __forceinline__ void store_one(char *p, float v)
{
    if constexpr (DT == kBf16)
        *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(v);
    else
        *reinterpret_cast<float *>(p) = v;
}

// Sums of 2^z and of 2^z z, z = c (x - ref).
struct Sums {
    float ref, s, w;

    __device__ __forceinline__ void rebase(float to, float c)
    {
        if (ref == neg_inf()) {  // nothing summed yet
            ref = to;
            return;
        }
        const float d = (ref - to) * c, f = exp2_fast(d);
        w = f > 0.0f ? (w + d * s) * f : w * f;  // (a NaN stays one)
        s *= f;
        ref = to;
    }
};

// The chunk's part of the sums; `low` = floor_of(ref).
template <int IN, bool ENT>
__device__ __forceinline__ void add_chunk(F2 &s2, F2 &w2, const Chunk<IN> &x, float ref, float low, float c)
{
    const F2 minus = f2(-ref, -ref), cc = f2(c, c);
    if (ENT && low == neg_inf()) {
#pragma unroll
        for (int i = 0; i < Chunk<IN>::kVals / 2; ++i) {
            float a, b;
            f2_split(f2_mul(f2_add(x.pair(i), minus), cc), a, b);
            const float ea = exp2_fast(a), eb = exp2_fast(b);
            s2 = f2_add(s2, f2(ea, eb));
            w2 = f2_add(w2, f2(ea > 0.0f ? ea * a : 0.0f, eb > 0.0f ? eb * b : 0.0f));
        }
        return;
    }
    Chunk<IN> y = x;
    if constexpr (ENT)
        y = x.raised(low);
#pragma unroll
    for (int i = 0; i < Chunk<IN>::kVals / 2; ++i) {
        const F2 z = f2_mul(f2_add(y.pair(i), minus), cc);
        float a, b;
        f2_split(z, a, b);
        const F2 e = f2(exp2_fast(a), exp2_fast(b));
        s2 = f2_add(s2, e);
        if constexpr (ENT)
            w2 = f2_fma(e, z, w2);
    }
}

// The next larger value; -inf gives the lowest finite one, inf none (a NaN).
__device__ __forceinline__ float next_above(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    return __uint_as_float((u >> 31) ? u - 1 : u + 1);
}

// Order of logits: by value, equal ones by index; a larger key comes first.
__device__ __forceinline__ unsigned long long key_of(float v, int index)
{
    uint32_t u = __float_as_uint(v + 0.0f);  // -0 equals 0
    u ^= (u >> 31) ? 0xFFFFFFFFu : 0x80000000u;
    return (static_cast<unsigned long long>(u) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(index));
}
__device__ __forceinline__ float key_value(unsigned long long key)
{
    uint32_t u = static_cast<uint32_t>(key >> 32);
    u ^= (u >> 31) ? 0x80000000u : 0xFFFFFFFFu;
    return __uint_as_float(u);
}

__device__ __forceinline__ uint32_t in_block(const void *p, uint32_t rank) { return map_to_cta(smem_addr(p), rank); }
__device__ __forceinline__ float ld_f32(uint32_t a)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_u32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long ld_u64(uint32_t a)
{
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(m) : "f"(v));
    return m;
}

// The k-th largest of the lanes' values.
__device__ __forceinline__ float warp_kth(float v, int k)
{
    float m = warp_max(v);
    for (int n = __popc(__ballot_sync(0xFFFFFFFFu, v == m)); n < k && m != neg_inf();
         n += __popc(__ballot_sync(0xFFFFFFFFu, v == m))) {
        v = v == m ? neg_inf() : v;
        m = warp_max(v);
    }
    return m;
}

// A row as a block sees it: whole chunks from a 32-byte boundary on, which the blocks of
// the cluster share, and up to 15 values before and after, one to a thread of the first
// block.
template <int IN>
struct Row {
    static constexpr int E = ElemBytes<IN>::value;
    const char *x;
    int head, chunks;
    int from, to;  // this block's chunks
    int extras;

    __device__ __forceinline__ Row(const char *row, int V, int rank, int log_blocks) : x(row)
    {
        head = static_cast<int>((32 - (reinterpret_cast<uintptr_t>(row) & 31)) & 31) / E;
        head = head < V ? head : V;
        chunks = (V - head) / Chunk<IN>::kVals;
        const int per = (chunks + (1 << log_blocks) - 1) >> log_blocks;
        from = rank * per < chunks ? rank * per : chunks;
        to = from + per < chunks ? from + per : chunks;
        extras = rank == 0 ? V - chunks * Chunk<IN>::kVals : 0;
    }
    __device__ __forceinline__ int first_of(int chunk) const { return head + chunk * Chunk<IN>::kVals; }
    __device__ __forceinline__ int extra(int i) const { return i < head ? i : i + chunks * Chunk<IN>::kVals; }
    __device__ __forceinline__ const char *at(int v) const { return x + static_cast<int64_t>(v) * E; }
    __device__ __forceinline__ float one(int v) const { return load_one<IN>(at(v)); }
};

// The first bytes of a later row into L2: blocks that start together end together, and
// HBM would idle through their last steps (4096 x 128256 BF16 with the 20 most probable
// 174 us, 179 without; 16 and 64 KB 177 and 173; with entropy 184, without 186, and 184 and 185).
__device__ __forceinline__ void fetch_ahead(const char *row, int64_t bytes)
{
    const int skip = static_cast<int>(-reinterpret_cast<uintptr_t>(row) & 15);
    const int size = static_cast<int>((bytes < kFetchAhead ? bytes : kFetchAhead) - skip) & ~15;
    if (size > 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(row + skip), "r"(size) : "memory");
}

// TOP: every thread keeps the maxima of its chunks, 2^log_group of them in one, and the
// groups whose maximum counts are what is listed, so that a long row's list is no longer than a
// short one's (1300 x 262144 FP32 with the 32 most probable 251 us; a list of their chunks
// overflowed, and the pass a token below took 11 ms).  SPLIT: a
// cluster of 2^log_blocks blocks shares a row; there are few rows then, so more chunks in
// flight count for more than more blocks on a multiprocessor (64 x 128256 with entropy and the
// 20 most probable: 9.4 us with four chunks and two blocks, 11.9 with two and four).
template <int IN, bool ENT, bool TOP, bool SPLIT>
__global__ void __launch_bounds__(kThreads, SPLIT ? 2 : 4) logprobs_kernel(const LogprobsParams p, int log_blocks, int log_group, int resident)
{
    extern __shared__ float maxima[];  // [kept][threads], TOP only
    __shared__ float warp_m[kWarps], warp_s[kWarps], warp_w[kWarps], warp_bound[kWarps];
    __shared__ float block_m, block_s, block_w, block_bound;
    __shared__ unsigned long long candidates[TOP ? kCandidates : 1];
    __shared__ unsigned long long warp_best[kWarps], list[32];
    __shared__ int warp_equal[kWarps];
    __shared__ uint32_t count, groups_found, group_list[TOP ? kGroupList : 1];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
    constexpr int kAhead = SPLIT ? 4 : 2;  // chunks of a thread in flight
    const int group = 1 << log_group, blocks = SPLIT ? 1 << log_blocks : 1, rank = SPLIT ? static_cast<int>(blockIdx.x) & (blocks - 1) : 0;
    const int64_t row = SPLIT ? blockIdx.x >> log_blocks : blockIdx.x;
    auto everybody = [&]() {
        if constexpr (SPLIT)
            cluster_sync();
        else
            __syncthreads();
    };
    const Row<IN> r(p.x + row * p.stride, static_cast<int>(p.V), rank, SPLIT ? log_blocks : 0);
    const float c = p.scale * kLog2E, step_up = kMargin / c;
    if (tid == 0)
        count = groups_found = 0;

    // ---- the pass over the row
    Sums a = {neg_inf(), 0.0f, 0.0f};
    float low = neg_inf(), own_max = neg_inf();
    F2 s2 = f2(0.0f, 0.0f), w2 = f2(0.0f, 0.0f);
    bool nan = false, real = false;
    float target_x = 0.0f;  // thread 0's
    // this thread's chunks
    const int mine = r.to - r.from > tid ? (r.to - r.from - tid + threads - 1) / threads : 0;
    float kept = neg_inf();
    int in_group = 0, keep = tid;
    auto take = [&](const Chunk<IN> &x) {
        float m = x.max();
        if (!(m <= a.ref + step_up)) {  // (also where the reference is still missing, and for a NaN)
            if (m != m) {
                nan = true;
                m = neg_inf();
#pragma unroll
                for (int i = 0; i < Chunk<IN>::kVals; ++i)
                    m = fmaxf(m, x.at(i));
            }
            if (m > a.ref) {
                float lo, hi;
                f2_split(s2, lo, hi);
                a.s = lo + hi;
                f2_split(w2, lo, hi);
                a.w = lo + hi;
                a.rebase(m, c);
                s2 = f2(a.s, 0.0f);
                w2 = f2(a.w, 0.0f);
                low = floor_of(m, c);
            }
        }
        own_max = fmaxf(own_max, m);
        if constexpr (TOP) {
            kept = fmaxf(kept, m);
            if (++in_group == group) {
                maxima[keep] = kept;
                keep += threads;
                kept = neg_inf();
                in_group = 0;
            }
        }
        if (a.ref != neg_inf())  // else every value is -inf and adds nothing
            add_chunk<IN, ENT>(s2, w2, x, a.ref, low, c);
    };
    {
        Chunk<IN> x[kAhead];
        const char *from = r.at(r.first_of(r.from + tid));
        const int64_t step = threads * 32;
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (j < mine)
                x[j].load(from + j * step);
        if (rank == 0 && tid == 0 && p.targets) {
            const int64_t t = p.targets64 ? static_cast<const int64_t *>(p.targets)[row]
                                          : static_cast<const int32_t *>(p.targets)[row];
            real = t >= 0 && t < p.V;
            if (real)
                target_x = r.one(static_cast<int>(t));
        }
        // the first reference: the largest value of the warp's first chunks
        float m = mine > 0 ? x[0].max() : neg_inf();
        a.ref = warp_max(m == m ? m : neg_inf());
        low = floor_of(a.ref, c);
        for (int i = 0; i < mine; i += kAhead) {
            from += kAhead * step;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (i + j >= mine)
                    break;
                const Chunk<IN> now = x[j];
                if (i + j + kAhead < mine)
                    x[j].load(from + j * step);
                take(now);
            }
        }
        if (TOP && in_group > 0)
            maxima[keep] = kept;
        float lo, hi;
        f2_split(s2, lo, hi);
        a.s = lo + hi;
        f2_split(w2, lo, hi);
        a.w = lo + hi;
    }
    if constexpr (!SPLIT) {
        if (tid == 0 && row + resident < p.rows)  // about the row that follows on this block's place
            fetch_ahead(p.x + (row + resident) * p.stride, p.V * ElemBytes<IN>::value);
    }
    if (tid < r.extras) {
        const float x = r.one(r.extra(tid));
        nan |= x != x;
        if (x > neg_inf()) {
            if (x > a.ref)
                a.rebase(x, c);
            const float z = (x - a.ref) * c, e = exp2_fast(z);
            a.s += e;
            a.w += e > 0.0f ? e * z : 0.0f;
            own_max = fmaxf(own_max, x);
        }
    }
    if (nan)
        a.s = a.w = __uint_as_float(0x7FC00000u);

    // ---- sums and bounds of the block
    const float m_warp = warp_max(own_max);
    if (m_warp != neg_inf())
        a.rebase(m_warp, c);
    a.s = warp_sum(a.s);
    if constexpr (ENT)
        a.w = warp_sum(a.w);
    // at least `each` threads of every warp reach the warp's bound, and `of` warps the block's
    const int need = TOP ? (p.top + blocks - 1) / blocks : 1;
    const int each = (need + warps - 1) / warps, of = (need + each - 1) / each;
    const float bound = TOP && each > 1 ? warp_kth(own_max, each) : m_warp;
    if (lane == 0) {
        warp_m[warp] = m_warp;
        warp_s[warp] = a.s;
        warp_w[warp] = a.w;
        warp_bound[warp] = bound;
    }
    __syncthreads();
    // the largest and the sums of as many parts as there are lanes, for all of them
    auto join = [&](Sums &b) {
        const float m = warp_max(b.ref);
        if (m != neg_inf())
            b.rebase(m, c);
        b.s = warp_sum(b.s);
        if constexpr (ENT)
            b.w = warp_sum(b.w);
        b.ref = m;
    };
    Sums b = {neg_inf(), 0.0f, 0.0f};
    if (warp == 0) {
        if (lane < warps)
            b = {warp_m[lane], warp_s[lane], warp_w[lane]};
        join(b);
        if (SPLIT && lane == 0) {
            block_m = b.ref;
            block_s = b.s;
            block_w = b.w;
        }
    }
    if (TOP && warp == warps - 1) {  // beside the first warp where there is another
        const float v = warp_kth(lane < warps ? warp_bound[lane] : neg_inf(), of);
        if (lane == 0)
            block_bound = v;
    }
    everybody();

    // ---- the row's sums
    float log_s = 0.0f, row_m = neg_inf();
    if (rank == 0 && warp == 0) {
        if constexpr (SPLIT) {
            b = {neg_inf(), 0.0f, 0.0f};
            if (lane < blocks) {
                b.ref = ld_f32(in_block(&block_m, lane));
                b.s = ld_f32(in_block(&block_s, lane));
                b.w = ld_f32(in_block(&block_w, lane));
            }
            join(b);
        }
        row_m = b.ref;
        log_s = logf(b.s);
        if (lane == 0) {
            // a row without a finite value: no token has a probability, and nothing is uncertain
            const bool none = row_m == neg_inf() && b.s == 0.0f;
            if (none)
                log_s = 0.0f;
            if (p.logprob)
                p.logprob[row] = !real ? 0.0f : none ? neg_inf() : (target_x - row_m) * p.scale - log_s;
            if (p.entropy)
                p.entropy[row] = none ? 0.0f : log_s - kLn2 * (b.w / b.s);
            if (p.stats)
                reinterpret_cast<float2 *>(p.stats)[row] = make_float2(row_m, log_s);
        }
        if constexpr (TOP) {
            if (lane == 0) {  // for the ranks below
                warp_m[0] = row_m;
                warp_s[0] = log_s;
            }
        }
    }
    if constexpr (!TOP) {
        if constexpr (SPLIT)
            cluster_sync();  // no block leaves while the first may still read its sums
        return;
    }

    // ---- the most probable tokens
    float least = block_bound;
    if constexpr (SPLIT) {
        least = ld_f32(in_block(&block_bound, lane & (blocks - 1)));  // a block a lane: one latency for all of them
#pragma unroll
        for (int o = kLogprobsCluster / 2; o > 0; o >>= 1)
            least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
    }
    // the row's candidates, in the first block, in any order: they are ranked by their keys
    const uint32_t to_count = in_block(&count, 0), to_list = in_block(candidates, 0);
    auto places = [&](uint32_t n) {
        if constexpr (SPLIT) {
            uint32_t at;
            asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(at) : "r"(to_count), "r"(n) : "memory");
            return at;
        } else {
            return atomicAdd(&count, n);
        }
    };
    auto put = [&](uint32_t at, float v, int index) {
        if (at >= kCandidates)
            return;
        if constexpr (SPLIT)
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to_list + at * 8), "l"(key_of(v, index)) : "memory");
        else
            candidates[at] = key_of(v, index);
    };
    auto offer = [&](float v, int index) { put(places(1), v, index); };
    // Offers the logits that reach `least`, or, `over`, those above it.
    auto collect = [&](bool over) {
        const float reach = over ? next_above(least) : fmaxf(least, -FLT_MAX);
        auto counts = [&](float v) { return v >= reach; };  // -inf never does
        // the sum of the lanes' up to this one
        auto up_to_lane = [&](uint32_t n) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, n, o);
                n += lane >= o ? v : 0;
            }
            return n;
        };
        // the groups of chunks whose maximum counts
        if (__any_sync(0xFFFFFFFFu, counts(own_max))) {
            uint32_t hits = 0;
            const int kept_n = (mine + group - 1) >> log_group;
#pragma unroll 8
            for (int i = 0; i < kept_n; ++i)
                hits |= static_cast<uint32_t>(counts(maxima[i * threads + tid])) << i;
            uint32_t at = up_to_lane(__popc(hits)), start = 0;
            if (lane == 31)
                start = atomicAdd(&groups_found, at);
            at += __shfl_sync(0xFFFFFFFFu, start, 31) - __popc(hits);
            for (; hits; hits &= hits - 1, ++at)
                if (at < kGroupList)
                    group_list[at] = tid + ((__ffs(hits) - 1) << log_group) * threads;  // its first chunk
        }
        __syncthreads();
        // their values: eight bytes a thread, two at a time
        if (groups_found > kGroupList) {
            if (tid == 0)  // too many for the list: so will the candidates be
                places(kCandidates + 1);
        } else {
            constexpr int kPart = Chunk<IN>::kVals / 4;
            const uint32_t parts = groups_found << (log_group + 2);
            for (uint32_t first = warp * 32; first < parts; first += 2 * threads) {
                uint32_t w[4], hits = 0;
                int index[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t i = first + lane + j * threads;
                    uint32_t chunk = 0xFFFFFFFFu;
                    if (i < parts)
                        chunk = SPLIT && log_group == 0 ? group_list[i >> 2]
                                                        : group_list[i >> (log_group + 2)] + ((i >> 2) & (group - 1)) * threads;
                    index[j] = -1;
                    if (chunk < static_cast<uint32_t>(r.to - r.from)) {
                        index[j] = r.first_of(r.from + chunk) + (i & 3) * kPart;
                        const uint2 v = *reinterpret_cast<const uint2 *>(r.at(index[j]));
                        w[2 * j] = v.x;
                        w[2 * j + 1] = v.y;
                    }
                }
                auto value = [&](uint32_t word, int n) {
                    return __uint_as_float(IN == kF32 ? word : (n & 1) ? (word & 0xFFFF0000u) : (word << 16));
                };
#pragma unroll
                for (int n = 0; n < 2 * kPart; ++n)
                    if (index[n / kPart] >= 0 && counts(value(w[n * 2 / kPart], n)))
                        hits |= 1u << n;
                if (!__any_sync(0xFFFFFFFFu, hits))
                    continue;
                uint32_t at = up_to_lane(__popc(hits)), start = 0;  // one addition for the warp's
                if (lane == 31)
                    start = places(at);
                at += __shfl_sync(0xFFFFFFFFu, start, 31) - __popc(hits);
                for (; hits; hits &= hits - 1, ++at) {
                    const int n = __ffs(hits) - 1, k = n * 2 / kPart;
                    put(at, value(k < 2 ? (k ? w[1] : w[0]) : (k == 2 ? w[2] : w[3]), n), (n < kPart ? index[0] : index[1]) + n % kPart);
                }
            }
        }
        if (tid < r.extras && counts(r.one(r.extra(tid))))
            offer(r.one(r.extra(tid)), r.extra(tid));
    };
    bool over = false;
    uint32_t n = 0;
    for (int tries = 0;; ++tries) {
        collect(over);
        if (over)
            break;
        everybody();
        n = SPLIT ? ld_u32(to_count) : count;
        if (n <= kCandidates)
            break;
        everybody();
        if (tid == 0)
            count = groups_found = 0;
        // The largest logits are next to each other (tokens of one range, the others masked), so that few warps hold
        // them: the `top`-th largest maximum of a block's threads is reached often enough by itself.
        over = true;
        if (tries == 0) {
            float *const all = reinterpret_cast<float *>(group_list);
            all[tid] = own_max;
            __syncthreads();
            int larger = 0;
            for (int i = 0; i < threads; ++i)
                larger += all[i] > own_max || (all[i] == own_max && i < tid);
            if (larger == p.top - 1)
                block_bound = own_max;
            everybody();
            float bound = block_bound;
            if constexpr (SPLIT)
                bound = warp_max(ld_f32(in_block(&block_bound, lane & (blocks - 1))));
            over = bound <= least;
            least = fmaxf(least, bound);
        }
        everybody();
    }
    if (over) {
        // Many equal logits (a mask of the type's lowest value): those above the bound, and each block's first ones of
        // those that equal it.
        if (tid < r.extras && r.one(r.extra(tid)) == least && least != neg_inf())
            offer(least, r.extra(tid));
        int found = 0;  // equal ones before this tile of chunks
        for (int i = 0; i * threads < r.to - r.from && found < p.top && least != neg_inf(); ++i) {
            const bool here = i < mine && maxima[(i >> log_group) * threads + tid] >= least;
            if (!__syncthreads_or(here))
                continue;
            uint32_t equal = 0;
            if (here) {
                Chunk<IN> x;
                x.load(r.at(r.first_of(r.from + i * threads + tid)));
#pragma unroll
                for (int j = 0; j < Chunk<IN>::kVals; ++j)
                    equal |= static_cast<uint32_t>(x.at(j) == least) << j;
            }
            int before = __popc(equal);  // and in the chunks before this one
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
                before += lane >= o ? v : 0;
            }
            if (lane == 31)
                warp_equal[warp] = before;
            __syncthreads();
            before += found - __popc(equal);
            for (int w = 0; w < warps; ++w) {
                before += w < warp ? warp_equal[w] : 0;
                found += warp_equal[w];
            }
            for (; equal && before < p.top; equal &= equal - 1, ++before)
                offer(least, r.first_of(r.from + i * threads + tid) + __ffs(equal) - 1);
            __syncthreads();
        }
        everybody();
        n = SPLIT ? ld_u32(to_count) : count;
    }
    if (n > kCandidates) {
        // Too many are above it (the largest of the row in few threads' chunks): every block finds its own best ones, one
        // at a time, and the first block ranks those.
        unsigned long long last = ~0ull;
        for (int k = 0; k < p.top; ++k) {
            unsigned long long best = 0;
            auto look = [&](float v, int index) {
                const unsigned long long key = key_of(v, index);
                if (v > neg_inf() && key < last && key > best)
                    best = key;
            };
            for (int chunk = r.from + tid; chunk < r.to; chunk += threads) {
                Chunk<IN> x;
                x.load(r.at(r.first_of(chunk)));
#pragma unroll
                for (int i = 0; i < Chunk<IN>::kVals; ++i)
                    look(x.at(i), r.first_of(chunk) + i);
            }
            if (tid < r.extras)
                look(r.one(r.extra(tid)), r.extra(tid));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const unsigned long long v = __shfl_xor_sync(0xFFFFFFFFu, best, o);
                best = v > best ? v : best;
            }
            if (lane == 0)
                warp_best[warp] = best;
            __syncthreads();
            for (int w = 0; w < warps; ++w)
                best = warp_best[w] > best ? warp_best[w] : best;
            if (tid == 0)
                list[k] = best;  // 0: there are no more
            last = best;
            __syncthreads();
        }
        everybody();
        n = static_cast<uint32_t>(p.top * blocks);
        if (rank == 0)
            for (uint32_t i = tid; i < n; i += threads)
                candidates[i] = ld_u64(in_block(list, i / p.top) + i % p.top * 8);
        __syncthreads();
    }
    __syncwarp();
    if constexpr (SPLIT)
        cluster_arrive();  // this block reads no other's memory any more
    if (rank == 0) {
        const float m = warp_m[0], ls = warp_s[0];
        int64_t *ids = p.top_ids + row * p.top;
        float *values = p.top_logprobs + row * p.top;
        for (uint32_t i = tid; i < n; i += threads) {
            const unsigned long long key = candidates[i];
            if (key == 0)
                continue;
            uint32_t larger = 0;
#pragma unroll 8
            for (uint32_t j = 0; j < n; ++j)
                larger += candidates[j] > key;
            if (larger < static_cast<uint32_t>(p.top)) {
                ids[larger] = 0xFFFFFFFFu - static_cast<uint32_t>(key);
                values[larger] = (key_value(key) - m) * p.scale - ls;
            }
        }
        // fewer than `top` tokens with a probability: the rest is -1
        uint32_t found = 0;
        for (uint32_t j = lane; j < n; j += 32)
            found += candidates[j] != 0;
        found = __reduce_add_sync(0xFFFFFFFFu, found);
        for (uint32_t i = found + tid; i < static_cast<uint32_t>(p.top); i += threads) {
            ids[i] = -1;
            values[i] = neg_inf();
        }
    }
    __syncwarp();
    if constexpr (SPLIT)
        cluster_wait();  // no block leaves while another may still read its memory
}

// ----------------------------------------------------------------- backward --
// Bound by HBM: 4096 x 128256 BF16 295 us (7.1 TB/s with what stays in L2), with entropy or
// without; 8192 x 1000 FP32 9.8 us; where logits and gradient start differently, 1000 x
// 50257 FP32 80 us instead of 60, BF16 81 instead of 32.
// A block takes kBackChunks chunks a thread of a row.  VECTOR: the row and its gradient
// start alike against 32-byte boundaries; else one value a thread at a time.
constexpr int kBackChunks = 2;
template <int IN>
__device__ __host__ __forceinline__ int64_t back_values(int threads)  // of a block
{
    return static_cast<int64_t>(threads) * kBackChunks * Chunk<IN>::kVals;
}

struct RowGrad {
    float m, c, shift;   // ln p = ln2 * t, t = (x - m) * c - shift
    float a, b;          // p * (a + b * t) is the gradient, apart from the target's own term
    float low;           // values are raised to it
    bool none;           // a row without a finite value

    __device__ __forceinline__ float at(float x) const
    {
        const float t = fmaf(x - m, c, -shift), p = exp2_fast(t);
        return none || p == 0.0f ? 0.0f : p * fmaf(b, t, a);
    }
};

template <int IN, bool ENT, bool VECTOR>
__global__ void __launch_bounds__(kThreads) logprobs_backward_kernel(const LogprobsBackParams p, uint32_t per_row)
{
    constexpr int E = ElemBytes<IN>::value;
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, threads = blockDim.x;
    const uint32_t part = blockIdx.x % per_row;
    const int64_t row = blockIdx.x / per_row, V = p.V;
    const char *x = p.x + row * p.stride;
    char *d = p.dlogits + row * p.dlogits_stride;
    const int64_t head = VECTOR ? min(static_cast<int64_t>(((32 - (reinterpret_cast<uintptr_t>(x) & 31)) & 31) / E), V) : 0;
    const int64_t chunks = VECTOR ? (V - head) / Chunk<IN>::kVals : 0;
    const int64_t c0 = static_cast<int64_t>(part) * threads * kBackChunks + tid;
    Chunk<IN> v[kBackChunks];
    if constexpr (VECTOR)
#pragma unroll
        for (int j = 0; j < kBackChunks; ++j)
            if (c0 + j * threads < chunks)
                v[j].load(x + (head + (c0 + j * threads) * Chunk<IN>::kVals) * E);
    const int64_t target = p.targets == nullptr ? -1
                           : p.targets64        ? static_cast<const int64_t *>(p.targets)[row]
                                                : static_cast<const int32_t *>(p.targets)[row];
    const bool real = target >= 0 && target < V;
    const float2 stats = reinterpret_cast<const float2 *>(p.stats)[row];
    const float g = real && p.dlogprob ? p.dlogprob[row] : 0.0f;
    const float h = ENT ? p.dentropy[row] : 0.0f;
    RowGrad r;
    r.m = stats.x;
    r.c = p.scale * kLog2E;
    r.shift = stats.y * kLog2E;
    r.a = ENT ? -(g + h * p.entropy[row]) * p.scale : -g * p.scale;
    r.b = -h * kLn2 * p.scale;
    r.low = floor_of(stats.x, r.c, fmaxf(1.0f, fabsf(r.b)));
    r.none = stats.x == neg_inf();
    const float peak = r.none ? 0.0f : g * p.scale;
    auto single = [&](int64_t i) {
        store_one<IN>(d + i * E, r.at(load_one<IN>(x + i * E)) + (i == target ? peak : 0.0f));
    };
    if constexpr (!VECTOR) {
        constexpr int kAhead = 8;  // values a thread has in flight
        const int64_t end = min(V, (part + 1) * back_values<IN>(threads));
        for (int64_t i = part * back_values<IN>(threads) + tid; i < end; i += kAhead * threads) {
            float one[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                one[j] = i + j * threads < end ? load_one<IN>(x + (i + j * threads) * E) : 0.0f;
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (i + j * threads < end)
                    store_one<IN>(d + (i + j * threads) * E, r.at(one[j]) + (i + j * threads == target ? peak : 0.0f));
        }
        return;
    }
    const F2 minus = f2(-r.m, -r.m), cc = f2(r.c, r.c), shift = f2(-r.shift, -r.shift), a2 = f2(r.a, r.a),
             b2 = f2(r.b, r.b);
#pragma unroll
    for (int j = 0; j < kBackChunks; ++j) {
        if (c0 + j * threads >= chunks)
            break;
        const int64_t k = head + (c0 + j * threads) * Chunk<IN>::kVals;
        float o[Chunk<IN>::kVals];
        if (r.none || r.low == neg_inf()) {
#pragma unroll
            for (int i = 0; i < Chunk<IN>::kVals; ++i)
                o[i] = r.at(v[j].at(i));
        } else {
            const Chunk<IN> y = ENT ? v[j].raised(r.low) : v[j];
#pragma unroll
            for (int i = 0; i < Chunk<IN>::kVals / 2; ++i) {
                const F2 t = f2_fma(f2_add(y.pair(i), minus), cc, shift);
                float lo, hi;
                f2_split(t, lo, hi);
                const F2 e = f2(exp2_fast(lo), exp2_fast(hi));
                f2_split(f2_mul(e, ENT ? f2_fma(b2, t, a2) : a2), o[2 * i], o[2 * i + 1]);
            }
        }
        if (target >= k && target < k + Chunk<IN>::kVals)
#pragma unroll
            for (int i = 0; i < Chunk<IN>::kVals; ++i)
                if (target == k + i)
                    o[i] += peak;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = IN == kBf16 ? pack_bf16(o[2 * i % Chunk<IN>::kVals], o[(2 * i + 1) % Chunk<IN>::kVals])
                               : __float_as_uint(o[i]);
        st_row32(d + k * E, w);
    }
    const int64_t extras = V - chunks * Chunk<IN>::kVals;
    if (part == 0 && tid < extras)
        single(tid < head ? tid : tid + chunks * Chunk<IN>::kVals);
}

// Threads of a block for long rows, such that as little of the machine idles as can be: 700 x 50257 FP32 with the 20 most
// probable 28.6 us in one wave of blocks of 192, 36.3 in a wave of 256 and a seventh of one.  In tenths of a row's time on a full multiprocessor: the full waves' rows, those of the last one, which takes no
// less than six tenths of a full one, and every wave's last steps.  After three waves blocks no longer end together
// (4096 x 128256 BF16 with the 20 most probable: on blocks of 96 192 us, 174 on those of 256).  Of 364 sizes (160 to 1824
// rows of 9000 to 262144 values, both types, with the 20 most probable and without) blocks of 256 throughout take 0.90 to
// 1.51 times this choice's time, 1.05 in the mean; the best of the five sizes 0.97 in the mean and 0.79 at the least.
int wave_threads(int64_t rows, int num_sms, int resident)
{
    int64_t least = INT64_MAX;
    int threads = kThreads;
    for (const int t : {256, 192, 160, 128, 96}) {
        const int64_t fit = resident / t, wave = fit * num_sms, full = rows / wave, rest = rows % wave;
        const int64_t last = rest == 0 ? 0 : std::max(10 * rest / num_sms, 6 * fit);
        const int64_t cost = 10 * fit * full + last + 5 * (full + (rest > 0));
        if (cost < least) {
            least = cost;
            threads = t;
        }
    }
    return threads;
}

template <int IN, bool ENT, bool TOP>
cudaError_t launch_rows(const LogprobsParams &p, int num_sms, int log_blocks, int threads, cudaStream_t s)
{
    cudaLaunchAttribute attr[1], both[2];
    const unsigned blocks = 1u << log_blocks;
    constexpr int resident = IN == kF32 && !ENT && !TOP ? 1280 : 1024;  // threads on a multiprocessor (46, up to 64 registers)
    if (log_blocks == 0 && threads == kThreads && p.rows <= 12ll * num_sms)
        threads = wave_threads(p.rows, num_sms, resident);
    // chunks of a thread at most (a row that starts off a 32-byte boundary may have one less)
    const int64_t chunks = (p.V / Chunk<IN>::kVals + blocks - 1) / blocks, mine = (chunks + threads - 1) / threads;
    // (smaller blocks, of which there are more on a multiprocessor, keep fewer: shared memory is L1's)
    const int most = threads >= kThreads ? kKeptMaxima : std::max(kKeptMaxima * threads / kThreads, kKeptMaxima / 2);
    int log_group = 0;
    while (mine > static_cast<int64_t>(most) << log_group)
        ++log_group;
    const int64_t kept = (mine + (1ll << log_group) - 1) >> log_group;
    const size_t smem = TOP ? static_cast<size_t>(kept) * threads * sizeof(float) : 0;
    cudaLaunchConfig_t cfg = row_launch(static_cast<unsigned>(p.rows * blocks), threads, smem, s, attr);
    if (blocks == 1)
        return cudaLaunchKernelEx(&cfg, logprobs_kernel<IN, ENT, TOP, false>, p, 0, log_group, num_sms * (resident / threads));
    both[0] = attr[0];
    both[1].id = cudaLaunchAttributeClusterDimension;
    both[1].val.clusterDim.x = blocks;
    both[1].val.clusterDim.y = 1;
    both[1].val.clusterDim.z = 1;
    cfg.attrs = both;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<IN, ENT, TOP, true>, p, log_blocks, log_group, 0);
}

template <int IN>
cudaError_t launch_forward(const LogprobsParams &p, int num_sms, cudaStream_t s)
{
    // few rows: blocks of a cluster share one, while each has at least two chunks a thread and all of them are resident
    // at once, two to a multiprocessor (100 x 128256 with the 20 most probable: 11.7 us on two blocks a row, 15.1 on four, where
    // a second wave is left)
    const int64_t chunks = p.V / Chunk<IN>::kVals;
    int log_blocks = 0;
    while ((1 << log_blocks) < kLogprobsCluster && p.rows << (log_blocks + 1) <= 2ll * num_sms &&
           chunks >= 4ll * kThreads << log_blocks)
        ++log_blocks;
    // short rows: fewer threads, down to a warp, of two chunks each; and where more rows are to be done than fit at once,
    // fewer still, up to sixteen chunks each, since a block's reductions are latency that other blocks have to cover
    // (8192 x 4096 BF16 12.6 us, 17.4 with two; 1446 x 10721 FP32 with the 20 most probable 15.0 us, 19.4 with six)
    int threads = kThreads;
    while (threads > 32 && chunks < 2ll * threads << log_blocks)
        threads /= 2;
    while (threads > 32 && chunks < 16ll * threads << log_blocks && p.rows * threads / 2 >= 1024ll * num_sms)
        threads /= 2;
    if (p.top > 0)
        return p.entropy ? launch_rows<IN, true, true>(p, num_sms, log_blocks, threads, s)
                         : launch_rows<IN, false, true>(p, num_sms, log_blocks, threads, s);
    return p.entropy ? launch_rows<IN, true, false>(p, num_sms, log_blocks, threads, s)
                     : launch_rows<IN, false, false>(p, num_sms, log_blocks, threads, s);
}

template <int IN, bool ENT>
cudaError_t launch_backward(const LogprobsBackParams &p, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    // every row and its gradient start alike where the first do and the rows' steps are alike
    const uintptr_t off = reinterpret_cast<uintptr_t>(p.x) - reinterpret_cast<uintptr_t>(p.dlogits);
    const bool vector = (off & 31) == 0 && (p.rows == 1 || ((p.stride - p.dlogits_stride) & 31) == 0);
    int threads = kThreads;
    while (threads > 64 && p.V <= back_values<IN>(threads / 2))  // short rows
        threads /= 2;
    const uint32_t per_row = static_cast<uint32_t>((p.V + back_values<IN>(threads) - 1) / back_values<IN>(threads));
    const cudaLaunchConfig_t cfg = row_launch(static_cast<unsigned>(p.rows * per_row), threads, 0, s, attr);
    return vector ? cudaLaunchKernelEx(&cfg, logprobs_backward_kernel<IN, ENT, true>, p, per_row)
                  : cudaLaunchKernelEx(&cfg, logprobs_backward_kernel<IN, ENT, false>, p, per_row);
}

}  // namespace

bool logprobs_fits(int64_t rows, int64_t V)
{
    return rows * ((V + back_values<kF32>(kThreads) - 1) / back_values<kF32>(kThreads)) < (1ll << 31) && rows * kLogprobsCluster < (1ll << 31);
}

cudaError_t launch_logprobs(const LogprobsParams &p, int in_dtype, int num_sms, cudaStream_t s)
{
    return in_dtype == kBf16 ? launch_forward<kBf16>(p, num_sms, s) : launch_forward<kF32>(p, num_sms, s);
}

cudaError_t launch_logprobs_backward(const LogprobsBackParams &p, int in_dtype, cudaStream_t s)
{
    if (in_dtype == kBf16)
        return p.dentropy ? launch_backward<kBf16, true>(p, s) : launch_backward<kBf16, false>(p, s);
    return p.dentropy ? launch_backward<kF32, true>(p, s) : launch_backward<kF32, false>(p, s);
}

}  // namespace mxg
