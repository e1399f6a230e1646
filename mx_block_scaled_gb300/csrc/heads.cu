// heads.cu -- RMS norm of query and key heads with the rotation of their
// positions, and its gradient.
//
//   n = x * rstd, rstd = 1/sqrt(mean(x^2) + eps) over a head;  y = R(position) (n * w)
//   g = R(-position) dy;  dx = rstd * (g * w - n * mean(g * w * n));  dw = sum over heads of g * n
//
// R turns the first `rotary` values of a head in pairs (a, b) -> (a cos - b sin, b cos + a sin),
// which are i and i + rotary/2, or 2i and 2i + 1.  A lane holds sixteen values of a
// head in which every pair is whole (two runs of eight), and their eight angles are
// the same eight consecutive ones in both orders: nothing but a sum crosses lanes.  A
// head takes a team of 1 to 32 lanes.
//
// One read and one write of the heads, two reads for the gradient.  16384 x 40 heads of
// 128 BF16 59 us (5.8 TB/s), their gradient at 8192 tokens 46 us (5.6 TB/s, 4 of it the
// second launch): instructions (300 and 370 for a warp's 512 values, issued in 72% of the
// cycles) nearly as much as HBM; FP32 10550 x 32 heads of 96 45 us, gradient of 4000 x 40
// of 128 43 us (0.87 and 0.85 of a copy).
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
    // values 2i and 2i + 1, and the other way round
    __device__ __forceinline__ F2 pair(int i) const { return f2(at(2 * i), at(2 * i + 1)); }
    __device__ __forceinline__ F2 swapped(int i) const { return f2(at(2 * i + 1), at(2 * i)); }
};

// Four pairs as eight values of type DT.
template <int DT>
__device__ __forceinline__ void store8(char *p, const F2 *pairs)
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f2_split(pairs[i], v[2 * i], v[2 * i + 1]);
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
            a = inside ? 16 * lane : 0;
            b = a + 8;
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

// Which weight a head takes (one past the last head: any that there is).
__device__ __forceinline__ bool is_query(const HeadsCommon &p, int h)
{
    return h < p.q_heads || p.q_heads == p.heads;
}

// Type of the weights of heads that are only rotated.
constexpr int kNoWeight = 0;

// A lane's sixteen weights, as pairs.
template <int WT>
struct Weights {
    F2 v[WT == kNoWeight ? 1 : 8];

    __device__ __forceinline__ void load(const HeadsCommon &p, const Place &at, bool query)
    {
        if constexpr (WT != kNoWeight) {
            constexpr int E = ElemBytes<WT>::value;
            const char *from = query ? p.q_weight : p.k_weight;
            Raw8<WT> a, b;
            a.load(from + at.a * E, at.inside);
            b.load(from + at.b * E, at.inside);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a.pair(i);
                v[4 + i] = b.pair(i);
            }
        }
    }
};

// A warp's walk over its share of the work: all steps (a group of neighbouring heads of
// a token, a head to each team) in order, split evenly over the warps of the grid.  What
// the steps ahead need is copied to the warp's own ring in shared memory (cp.async): the
// values of TENSORS tensors, rstd (TENSORS 2), and at a token's first step its angles,
// whose address waits for the token's position.  A warp that loads a token's heads into
// registers instead pays for that chain of latencies at every token.

__device__ __forceinline__ void cp_async16(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t to, const void *from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void lds16(uint32_t from, uint32_t *r)
{
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(from)
                 : "memory");
}

template <int IN, int TENSORS>
struct Ring {
    static constexpr int E = ElemBytes<IN>::value;
    static constexpr int kPieces = E / 2;             // 16-byte pieces of a run of eight
    static constexpr int kDepth = IN == kBf16 ? 4 : 2;  // stages, a power of two: more bytes a stage, fewer of them
    // heads of a group as they are in memory, then their rstd
    static __device__ __host__ __forceinline__ int stage_bytes(int team, int D)
    {
        return TENSORS * (32 / team) * D * E + (TENSORS == 2 ? 32 * 4 : 0);
    }
    // stages and angles (16 floats a member, a slot for every token under way) of a warp
    static __device__ __host__ __forceinline__ int bytes(int team, int D)
    {
        return kDepth * (stage_bytes(team, D) + team * 64);
    }

    const HeadsCommon &p;
    const Place at;
    const int team, member, mine, side;        // mine: the team's head of a group
    const int to_b;                            // bytes from a lane's first run to its second
    const int stage_size, tensor_size;         // bytes of a stage, of one tensor in it
    const uint32_t own, angles;                // this team's head in stage 0; the angle slots
    const uint32_t own_rstd;                   // its rstd in stage 0
    const char *const other;                   // TENSORS 2: dy
    const int64_t other_token, other_head;
    const float *const rstd;
    int left;                                  // steps to finish
    int64_t token;                             // of the current step
    int head, stage, slot;                     // head: the team's
    // the copying side: the next step's token, head and where its values are
    int64_t f_token, f_position;
    int f_head, f_stage, f_slot;
    const char *f_x, *f_other;
    const float *f_rstd;
    uint32_t real;                             // bit d: the token of angle slot d has a position of the table

    __device__ __forceinline__ int64_t position_of(int64_t t) const
    {
        if (!p.rope || t >= p.tokens)
            return 0;
        return p.positions64 ? static_cast<const int64_t *>(p.positions)[t] : static_cast<const int32_t *>(p.positions)[t];
    }

    __device__ __forceinline__ Ring(const HeadsCommon &params, const Place &place, int team_size, uint32_t smem,
                                    const char *other_p, int64_t other_t, int64_t other_h, const float *rstd_p)
        : p(params), at(place), team(team_size), member(threadIdx.x & (team_size - 1)),
          mine((threadIdx.x & 31) / team_size), side(32 / team_size), to_b((place.b - place.a) * E),
          stage_size(stage_bytes(team_size, p.D)), tensor_size(side * p.D * E),
          own(smem + (threadIdx.x >> 5) * bytes(team_size, p.D) + mine * p.D * E),
          angles(smem + (threadIdx.x >> 5) * bytes(team_size, p.D) + kDepth * stage_size),
          own_rstd(smem + (threadIdx.x >> 5) * bytes(team_size, p.D) + TENSORS * tensor_size + mine * 4),
          other(other_p), other_token(other_t), other_head(other_h), rstd(rstd_p)
    {
        const int64_t groups = (p.heads + side - 1) / side, all = p.tokens * groups;
        const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
        const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
        const int64_t each = all / warps, more = all % warps;  // the first `more` warps have one step more
        const int64_t u0 = w * each + (w < more ? w : more);
        left = static_cast<int>(each) + (w < more ? 1 : 0);
        token = f_token = u0 / groups;
        head = f_head = static_cast<int>(u0 - token * groups) * side + mine;
        stage = slot = f_stage = f_slot = 0;
        real = 0;
        f_position = left > 0 ? position_of(f_token) : 0;
        place_token();
#pragma unroll
        for (int d = 0; d < kDepth - 1; ++d)
            fetch(d < left, d == 0);  // (the first heads are not to wait for their token's position)
    }

    // a 16-byte piece of this member's angles; the members' pieces lie side by side, which their banks need
    __device__ __forceinline__ uint32_t angle_at(int d, int piece) const
    {
        return angles + ((d * 4 + piece) * team + member) * 16;
    }

    // a head by its team's lanes, neighbouring pieces by neighbouring lanes; `from`: this lane's first
    __device__ __forceinline__ void copy(uint32_t to, const char *from) const
    {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if ((i * team + member) * 16 < p.D * E)
                cp_async16(to + (i * team + member) * 16, from + i * team * 16);
    }

    // The copying side comes to a token: where its heads are.
    __device__ __forceinline__ void place_token()
    {
        f_x = p.x + f_token * p.x_token + f_head * p.x_head + member * 16;
        if constexpr (TENSORS == 2) {
            f_other = other + f_token * other_token + f_head * other_head + member * 16;
            f_rstd = rstd + f_token * p.heads + f_head;
        }
    }
    // And its angles.
    __device__ __forceinline__ void turn_token()
    {
        const int64_t position = f_position;
        const bool good = !p.rope || (position >= 0 && position < p.rope_rows);
        real = (real & ~(1u << f_slot)) | (static_cast<uint32_t>(good) << f_slot);
        if (p.rope && good && at.turned && mine == 0) {
            const float *row = p.rope + position * p.rotary + at.angle;
            cp_async16(angle_at(f_slot, 0), row);
            cp_async16(angle_at(f_slot, 1), row + 4);
            cp_async16(angle_at(f_slot, 2), row + p.rotary / 2);
            cp_async16(angle_at(f_slot, 3), row + p.rotary / 2 + 4);
        }
        f_position = position_of(f_token + 1);
        f_slot = (f_slot + 1) & (kDepth - 1);
    }

    __device__ __forceinline__ void fetch(bool any, bool first = false)
    {
        if (any) {
            if (!first && f_head - mine >= p.heads) {  // warp-uniform
                f_head = mine;
                ++f_token;
                place_token();
                turn_token();
            }
            if (f_head < p.heads) {
                copy(own + f_stage * stage_size, f_x);
                if constexpr (TENSORS == 2) {
                    copy(own + f_stage * stage_size + tensor_size, f_other);
                    if (member == 0)
                        cp_async4(own_rstd + f_stage * stage_size, f_rstd);
                }
            }
            if (first)
                turn_token();
            f_head += side;
            f_x += side * p.x_head;
            if constexpr (TENSORS == 2) {
                f_other += side * other_head;
                f_rstd += side;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        f_stage = (f_stage + 1) & (kDepth - 1);
    }

    // Makes the current step's copies visible and starts those of a later one; false: no step is left.
    __device__ __forceinline__ bool ready(bool &good)
    {
        if (left == 0)
            return false;
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
        __syncwarp();  // the others' copies have landed too, and nobody reads the stage that is refilled now
        good = (real >> slot) & 1;
        fetch(left >= kDepth);
        return true;
    }
    __device__ __forceinline__ bool live() const { return at.inside && head < p.heads; }
    // The current step's two runs of a tensor (whatever the memory holds where there are none).
    __device__ __forceinline__ void take(Raw8<IN> &a, Raw8<IN> &b, int tensor) const
    {
        const uint32_t from = own + stage * stage_size + tensor * tensor_size + at.a * E;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            lds16(from + 16 * i, a.r + 4 * i);
            lds16(from + to_b + 16 * i, b.r + 4 * i);
        }
    }
    __device__ __forceinline__ float take_rstd() const
    {
        float v;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(own_rstd + stage * stage_size) : "memory");
        return v;
    }
    // cosines (0..7) and sines (8..15) of this lane's angles (a turned lane's; whatever the memory holds where the
    // position is none of the table's)
    __device__ __forceinline__ void take_angles(float (&c)[16]) const
    {
        uint32_t r[16];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            lds16(angle_at(slot, i), r + 4 * i);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            c[i] = __uint_as_float(r[i]);
    }
    // On to the next step; true: it is another token's.
    __device__ __forceinline__ bool step()
    {
        --left;
        head += side;
        stage = (stage + 1) & (kDepth - 1);
        if (head - mine < p.heads)
            return false;
        head = mine;
        ++token;
        slot = (slot + 1) & (kDepth - 1);
        return true;
    }
};

// Pairs (a, b) -> (a cos - b sin, b cos + a sin), of the runs v[0..3] and v[4..7]; INVERSE: by minus the angles.
template <bool INTERLEAVED, bool INVERSE>
__device__ __forceinline__ void turn(F2 (&v)[8], const float (&c)[16])
{
    if constexpr (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float lo, hi;
            f2_split(v[i], lo, hi);
            const float sn = c[8 + i];
            v[i] = f2_fma(f2(hi, lo), INVERSE ? f2(sn, -sn) : f2(-sn, sn), f2_mul(v[i], f2(c[i], c[i])));
        }
    } else {
        const F2 minus = f2(-1.0f, -1.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F2 cs = f2(c[2 * i], c[2 * i + 1]), sn = f2(c[8 + 2 * i], c[9 + 2 * i]), neg = f2_mul(sn, minus);
            const F2 a = v[i], b = v[4 + i];
            v[i] = f2_fma(b, INVERSE ? sn : neg, f2_mul(a, cs));
            v[4 + i] = f2_fma(a, INVERSE ? neg : sn, f2_mul(b, cs));
        }
    }
}

// ------------------------------------------------------------------ forward --
constexpr int kForwardPerSm = 5;

// (and, INVERSE and without weights, the gradient of the rotation alone)
template <int IN, int WT, bool INTERLEAVED, bool INVERSE>
__global__ void __launch_bounds__(kThreads, kForwardPerSm) heads_kernel(const HeadsParams p, int team)
{
    constexpr int E = ElemBytes<IN>::value;
    extern __shared__ __align__(16) char heads_smem[];
    griddep_launch_dependents();
    griddep_wait();
    const Place at((threadIdx.x & 31) & (team - 1), p.D, p.rotary, INTERLEAVED);
    Ring<IN, 1> ring(p, at, team, smem_addr(heads_smem), nullptr, 0, 0, nullptr);
    const float inv_d = 1.0f / static_cast<float>(p.D);
    const bool leads = ring.member == 0 && p.rstd != nullptr;
    bool query = is_query(p, ring.head);
    Weights<WT> w;
    w.load(p, at, query);
    char *y = p.y + ring.token * p.y_token + ring.head * p.y_head + at.a * E;
    const int64_t y_step = ring.side * p.y_head;
    for (bool good; ring.ready(good);) {
        const int h = ring.head;
        Raw8<IN> a, b;
        ring.take(a, b, 0);
        F2 v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a.pair(i);
            v[4 + i] = b.pair(i);
        }
        if constexpr (WT != kNoWeight) {
            F2 ss2 = f2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss2 = f2_fma(v[i], v[i], ss2);
            float lo, hi;
            f2_split(ss2, lo, hi);
            const float rstd = rsqrtf(team_sum(at.inside ? lo + hi : 0.0f, team) * inv_d + p.eps);
            if (leads && h < p.heads)
                p.rstd[ring.token * p.heads + h] = good ? rstd : 0.0f;
            if (query != is_query(p, h)) {
                query = is_query(p, h);
                w.load(p, at, query);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = f2_mul(f2_mul(v[i], f2(rstd, rstd)), w.v[i]);
        }
        if (at.turned) {  // values that are not turned have no partner
            float c[16];
            ring.take_angles(c);
            turn<INTERLEAVED, INVERSE>(v, c);
        }
        if (!good)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = f2(0.0f, 0.0f);
        if (ring.live()) {
            store8<IN>(y, v);
            store8<IN>(y + ring.to_b, v + 4);
        }
        y += y_step;
        if (ring.step())
            y = p.y + ring.token * p.y_token + ring.head * p.y_head + at.a * E;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ----------------------------------------------------------------- backward --
// The same walk with dy, x and rstd.  A warp keeps the sums for both weights in
// registers; a block leaves its sums in partial[block][query, key][D], or, `joined`, for
// its cluster's first block.
template <int IN, int WT, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kHeadsBackPerSm) heads_backward_kernel(const HeadsBackParams p, int team, bool joined)
{
    constexpr int E = ElemBytes<IN>::value;
    extern __shared__ __align__(16) char heads_smem[];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Place at(lane & (team - 1), p.D, p.rotary, INTERLEAVED);
    Ring<IN, 2> ring(p, at, team, smem_addr(heads_smem), p.dy, p.dy_token, p.dy_head, p.rstd);
    const float inv_d = 1.0f / static_cast<float>(p.D);
    F2 dq[8], dk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        dq[i] = dk[i] = f2(0.0f, 0.0f);
    bool query = is_query(p, ring.head);
    Weights<WT> w;
    w.load(p, at, query);
    char *dx = p.dx + ring.token * p.dx_token + ring.head * p.dx_head + at.a * E;
    const int64_t dx_step = ring.side * p.dx_head;
    for (bool good; ring.ready(good);) {
        const int h = ring.head;
        Raw8<IN> xa, xb, ga, gb;
        ring.take(xa, xb, 0);
        ring.take(ga, gb, 1);
        float rstd = ring.take_rstd();
        F2 g[8], n[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            g[i] = ga.pair(i);
            g[4 + i] = gb.pair(i);
            n[i] = f2_mul(xa.pair(i), f2(rstd, rstd));
            n[4 + i] = f2_mul(xb.pair(i), f2(rstd, rstd));
        }
        if (at.turned) {  // values that are not turned have no partner
            float c[16];
            ring.take_angles(c);
            turn<INTERLEAVED, true>(g, c);
        }
        if (__any_sync(0xFFFFFFFFu, !good || !ring.live()))  // what is not there counts nothing, whatever the memory holds
            if (!good || !ring.live()) {
                rstd = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    g[i] = n[i] = f2(0.0f, 0.0f);
            }
        if (query != is_query(p, h)) {
            query = is_query(p, h);
            w.load(p, at, query);
        }
        F2 gw[8], dot2 = f2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            gw[i] = f2_mul(g[i], w.v[i]);
            dot2 = f2_fma(gw[i], n[i], dot2);
        }
        float lo, hi;
        f2_split(dot2, lo, hi);
        const float dot = team_sum(lo + hi, team) * -inv_d;
        if (query) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                dq[i] = f2_fma(g[i], n[i], dq[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                dk[i] = f2_fma(g[i], n[i], dk[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            gw[i] = f2_mul(f2_fma(n[i], f2(dot, dot), gw[i]), f2(rstd, rstd));
        if (!good)  // (a weight may be infinite)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                gw[i] = f2(0.0f, 0.0f);
        if (ring.live()) {
            store8<IN>(dx, gw);
            store8<IN>(dx + ring.to_b, gw + 4);
        }
        dx += dx_step;
        if (ring.step())
            dx = p.dx + ring.token * p.dx_token + ring.head * p.dx_head + at.a * E;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the rings are done with: the sums take their place
    float *const sums = reinterpret_cast<float *>(heads_smem);  // [kWarps][2][D]
    // over the teams of the warp, then over the warps in order
    float q_sum[16], k_sum[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f2_split(dq[i], q_sum[2 * i], q_sum[2 * i + 1]);
        f2_split(dk[i], k_sum[2 * i], k_sum[2 * i + 1]);
    }
    for (int o = team; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            q_sum[i] += __shfl_xor_sync(0xFFFFFFFFu, q_sum[i], o);
            k_sum[i] += __shfl_xor_sync(0xFFFFFFFFu, k_sum[i], o);
        }
    if (lane < team && at.inside) {
        float *out = sums + warp * 2 * p.D;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            out[at.a + i] = q_sum[i];
            out[at.b + i] = q_sum[8 + i];
            out[p.D + at.a + i] = k_sum[i];
            out[p.D + at.b + i] = k_sum[8 + i];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            v += sums[w * 2 * p.D + i];
        if (joined)
            sums[i] = v;  // its own place
        else
            p.partial[static_cast<int64_t>(blockIdx.x) * 2 * p.D + i] = v;
    }
    if (!joined)
        return;
    cluster_sync();  // the grid is one cluster: its first block adds the others' sums
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) {
            float v = 0.0f;
            for (uint32_t b = 0; b < gridDim.x; ++b) {
                float o;
                asm volatile("ld.shared::cluster.f32 %0, [%1];"
                             : "=f"(o)
                             : "r"(map_to_cta(smem_addr(sums + i), b))
                             : "memory");
                v += o;
            }
            float *out = i < p.D ? p.dq_weight : p.dk_weight;
            if (out)
                out[i < p.D ? i : i - p.D] = v;
        }
    cluster_sync();  // no block leaves before its sums are read
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

int64_t steps_of(int64_t tokens, int heads, int D)
{
    const int side = 32 / team_of(D);
    return tokens * ((heads + side - 1) / side);
}

// Blocks that the work fills, at most those that are on the multiprocessors at once.
int64_t blocks_of(int64_t tokens, int heads, int D, int64_t resident)
{
    const int64_t blocks = (steps_of(tokens, heads, D) + kWarps - 1) / kWarps;
    return blocks < resident ? blocks : resident;
}

// Blocks of a gradient that is one cluster, 0 where it is not: up to two steps a warp (with four, 108 steps take 7.2 us
// and two launches 4.9, but the host 3 us more for the second).
int64_t joined_blocks(int64_t tokens, int heads, int D)
{
    constexpr int64_t kCluster = 8, kSteps = 2 * kWarps;
    const int64_t steps = steps_of(tokens, heads, D);
    return steps <= kCluster * kSteps ? (steps + kSteps - 1) / kSteps : 0;
}

constexpr int kRingBytes = 216 * 1024;  // shared memory of an SM's rings
constexpr int kMostSmem = 96 * 1024;    // of a block; D = 512 in BF16, the largest, takes 66 KB

template <int IN, int WT>
cudaError_t prepare_kernels()
{
    constexpr auto kAttr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    constexpr int kForward = kMostSmem, kBackward = kMostSmem;
    cudaError_t e = cudaFuncSetAttribute(heads_kernel<IN, WT, false, false>, kAttr, kForward);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(heads_kernel<IN, WT, true, false>, kAttr, kForward);
    if constexpr (WT == kNoWeight) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(heads_kernel<IN, WT, false, true>, kAttr, kForward);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(heads_kernel<IN, WT, true, true>, kAttr, kForward);
    } else {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(heads_backward_kernel<IN, WT, false>, kAttr, kBackward);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(heads_backward_kernel<IN, WT, true>, kAttr, kBackward);
    }
    return e;
}

template <int IN, int WT>
cudaError_t launch_forward(const HeadsParams &p, bool interleaved, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const int team = team_of(p.D), smem = kWarps * Ring<IN, 1>::bytes(team, p.D), fit = kRingBytes / smem;
    const int64_t blocks = blocks_of(p.tokens, p.heads, p.D, static_cast<int64_t>(num_sms) * (fit < kForwardPerSm ? fit : kForwardPerSm));
    const cudaLaunchConfig_t cfg =
        row_launch(static_cast<unsigned>(blocks), kThreads, static_cast<size_t>(smem), s, attr);
    if constexpr (WT == kNoWeight)
        if (p.inverse)
            return interleaved ? cudaLaunchKernelEx(&cfg, heads_kernel<IN, WT, true, true>, p, team)
                               : cudaLaunchKernelEx(&cfg, heads_kernel<IN, WT, false, true>, p, team);
    return interleaved ? cudaLaunchKernelEx(&cfg, heads_kernel<IN, WT, true, false>, p, team)
                       : cudaLaunchKernelEx(&cfg, heads_kernel<IN, WT, false, false>, p, team);
}

template <int IN, int WT>
cudaError_t launch_backward(const HeadsBackParams &p, bool interleaved, int num_sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const int team = team_of(p.D), smem = kWarps * Ring<IN, 2>::bytes(team, p.D);  // more than the sums need: 8 D a warp
    const int64_t joined = joined_blocks(p.tokens, p.heads, p.D);
    cudaLaunchConfig_t cfg;
    if (joined > 0) {
        cudaLaunchAttribute both[2];
        cfg = row_launch(static_cast<unsigned>(joined), kThreads, static_cast<size_t>(smem), s, attr);
        both[0] = attr[0];
        both[1].id = cudaLaunchAttributeClusterDimension;
        both[1].val.clusterDim.x = static_cast<unsigned>(joined);
        both[1].val.clusterDim.y = 1;
        both[1].val.clusterDim.z = 1;
        cfg.attrs = both;
        cfg.numAttrs = 2;
        return interleaved ? cudaLaunchKernelEx(&cfg, heads_backward_kernel<IN, WT, true>, p, team, true)
                           : cudaLaunchKernelEx(&cfg, heads_backward_kernel<IN, WT, false>, p, team, true);
    }
    const int sms = num_sms < kHeadsBackSms ? num_sms : kHeadsBackSms, fit = kRingBytes / smem;
    const int64_t blocks = blocks_of(p.tokens, p.heads, p.D,
                                     static_cast<int64_t>(sms) * (fit < kHeadsBackPerSm ? fit : kHeadsBackPerSm));
    cfg = row_launch(static_cast<unsigned>(blocks), kThreads, static_cast<size_t>(smem), s, attr);
    const cudaError_t e = interleaved ? cudaLaunchKernelEx(&cfg, heads_backward_kernel<IN, WT, true>, p, team, false)
                                      : cudaLaunchKernelEx(&cfg, heads_backward_kernel<IN, WT, false>, p, team, false);
    if (e != cudaSuccess)
        return e;
    cfg = row_launch(static_cast<unsigned>(p.D / 16), 32 * kSlices, 0, s, attr);
    return cudaLaunchKernelEx(&cfg, heads_dweight_kernel, static_cast<const float *>(p.partial),
                              static_cast<int>(blocks), p.D, p.dq_weight, p.dk_weight);
}

}  // namespace

cudaError_t prepare_heads()
{
    cudaError_t e = prepare_kernels<kBf16, kNoWeight>();
    if (e == cudaSuccess)
        e = prepare_kernels<kBf16, kBf16>();
    if (e == cudaSuccess)
        e = prepare_kernels<kBf16, kF32>();
    if (e == cudaSuccess)
        e = prepare_kernels<kF32, kNoWeight>();
    if (e == cudaSuccess)
        e = prepare_kernels<kF32, kBf16>();
    return e == cudaSuccess ? prepare_kernels<kF32, kF32>() : e;
}

int64_t heads_back_blocks(int64_t tokens, int heads, int D)
{
    return joined_blocks(tokens, heads, D) > 0
               ? 0
               : blocks_of(tokens, heads, D, static_cast<int64_t>(kHeadsBackSms) * kHeadsBackPerSm);
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
