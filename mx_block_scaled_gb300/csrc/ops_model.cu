// ops_model.cu -- C ABI of the row operators at a model's ends and between its
// products (embedding, norm and rotation of heads, log probabilities, gradient norm
// and clipping): argument checks and launches.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "mx_block.cuh"
#include "mxgemm.h"
#include "ops.h"
#include "ops_check.h"

namespace {

using namespace mxg;

bool known_ids(int id_bytes) { return id_bytes == 4 || id_bytes == 8; }

// The kernels take exponents to base 2: scale * log2(e) is an FP32 number too.
bool scale_ok(float scale) { return scale > 0.0f && std::isfinite(scale * 1.4426950408889634f); }

// Rows of logits start where their type allows.
bool logits_shape_ok(int64_t stride, int64_t rows, int64_t V)
{
    return rows == 1 || (stride >= V && stride <= (1ll << 40));
}

// One vector [tokens, heads, D] with its strides in elements.
struct Heads {
    const void *p;
    int64_t token, head;
};

// Heads do not overlap: a token's heads lie inside its step, or a head's tokens inside the head's.
bool heads_shape_ok(const Heads &h, int64_t tokens, int64_t heads, int64_t D)
{
    constexpr int64_t kMost = 1ll << 40;
    if (!h.p)
        return true;
    if ((tokens > 1 && (h.token < D || h.token > kMost)) || (heads > 1 && (h.head < D || h.head > kMost)))
        return false;
    using Wide = __int128;  // 2^31 steps of 2^40 elements
    return tokens == 1 || heads == 1 || h.token >= static_cast<Wide>(heads - 1) * h.head + D ||
           h.head >= static_cast<Wide>(tokens - 1) * h.token + D;
}

bool heads_align_ok(const Heads &h, int64_t tokens, int64_t heads, int64_t elem)
{
    return !h.p || (aligned(h.p, 32) && (tokens == 1 || h.token * elem % 32 == 0) &&
                    (heads == 1 || h.head * elem % 32 == 0));
}

Span heads_span(const Heads &h, int64_t tokens, int64_t heads, int64_t D, int64_t elem)
{
    const int64_t token = tokens > 1 ? h.token : 0, head = heads > 1 ? h.head : 0;
    return {h.p, tokens, token * elem, ((heads - 1) * head + D) * elem};
}

bool same_heads(const Heads &a, const Heads &b, int64_t tokens, int64_t heads)
{
    return a.p == b.p && (tokens == 1 || a.token == b.token) && (heads == 1 || a.head == b.head);
}

// Checks of the sizes and the angles that both directions share.
int check_heads(int in_dtype, int weight_dtype, bool norm, int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t D,
                const float *rope, int64_t rope_rows, int64_t rotary, const void *positions, int position_bytes,
                uint32_t flags)
{
    if (!known_dtype(in_dtype) || (norm && !known_dtype(weight_dtype)) || (flags & ~MXGEMM_ROPE_INTERLEAVED))
        return MXGEMM_ERR_ARG;
    if ((rope == nullptr) != (positions == nullptr) || (rope && !known_ids(position_bytes)) || (!norm && !rope))
        return MXGEMM_ERR_ARG;
    if (tokens < 1 || tokens > kMaxRows || q_heads < 0 || k_heads < 0 || q_heads + k_heads < 1 ||
        q_heads > (1 << 20) || k_heads > (1 << 20) || D < 16 || D % 16 != 0 || D > kMaxCols)
        return MXGEMM_ERR_SHAPE;
    if (rope && (rope_rows < 1 || rope_rows > kMaxRows || rotary < 16 || rotary % 16 != 0 || rotary > D))
        return MXGEMM_ERR_SHAPE;
    if (!aligned(rope, 32) || (rope && !aligned(positions, static_cast<unsigned>(position_bytes))))
        return MXGEMM_ERR_ALIGN;
    if (D > kHeadsMaxDim || tokens * (q_heads + k_heads) > kMaxRows)
        return MXGEMM_ERR_UNSUPPORTED;
    return MXGEMM_OK;
}

void set_heads(HeadsCommon &p, int64_t e, int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t D, const Heads &x,
               const void *q_weight, const void *k_weight, const float *rope, int64_t rope_rows, int64_t rotary,
               const void *positions, int position_bytes)
{
    p.tokens = tokens;
    p.heads = static_cast<int>(q_heads + k_heads);
    p.q_heads = static_cast<int>(q_heads);
    p.D = static_cast<int>(D);
    p.rotary = rope ? static_cast<int>(rotary) : 0;
    p.q_weight = bytes(q_weight);
    p.k_weight = bytes(k_weight);
    p.rope = rope;
    p.rope_rows = rope_rows;
    p.positions = positions;
    p.positions64 = position_bytes == 8;
    p.x = bytes(x.p);
    p.x_token = x.token * e;
    p.x_head = x.head * e;
}

// A call's tensors as the kernels take them.
int read_grads(std::vector<GradTensor> &t, int64_t n, const void *const *grads, const int64_t *sizes,
               const int *dtypes, void *const *out, const int *out_dtypes)
{
    if (n < 0 || n > (1 << 20))
        return MXGEMM_ERR_SHAPE;
    if (n > 0 && (!grads || !sizes || !dtypes || (out != nullptr) != (out_dtypes != nullptr)))
        return MXGEMM_ERR_ARG;
    t.resize(static_cast<size_t>(n));
    for (int64_t i = 0; i < n; ++i) {
        GradTensor &g = t[i];
        const int to = out ? out_dtypes[i] : dtypes[i];
        const int64_t count = sizes[i];
        g.src = grads[i];
        g.dst = out ? out[i] : const_cast<void *>(grads[i]);
        if (count < 0 || count > (1ll << 40))
            return MXGEMM_ERR_SHAPE;
        if (!known_dtype(dtypes[i]) || !known_dtype(to) || (count > 0 && (!g.src || !g.dst)))
            return MXGEMM_ERR_ARG;
        if (!aligned(g.src, static_cast<unsigned>(elem_bytes(dtypes[i]))) ||
            !aligned(g.dst, static_cast<unsigned>(elem_bytes(to))))
            return MXGEMM_ERR_ALIGN;
        const uint32_t flags = (dtypes[i] == MXGEMM_IN_BF16 ? kGradSrcBf16 : 0) |
                               (to == MXGEMM_IN_BF16 ? kGradDstBf16 : 0) | (aligned(g.src, 32) ? kGradSrcVector : 0) |
                               (aligned(g.dst, 32) ? kGradDstVector : 0);
        g.n_flags = count << kGradFlagBits | flags;
    }
    return grads_fit(t.data(), n) ? MXGEMM_OK : MXGEMM_ERR_UNSUPPORTED;
}

struct Bytes {
    uintptr_t from, to;
    bool operator<(const Bytes &o) const { return from < o.from; }
};

// In the order of their addresses: an allocator leaves a few ascending runs, which are merged.
void sort_bytes(std::vector<Bytes> &v)
{
    constexpr size_t kRuns = 16;
    size_t run[kRuns + 1] = {0}, runs = 0;  // run[i] .. run[i + 1]: ascending
    for (size_t i = 1; i <= v.size(); ++i)
        if (i == v.size() || v[i] < v[i - 1]) {
            if (runs == kRuns) {
                std::sort(v.begin(), v.end());
                return;
            }
            run[++runs] = i;
        }
    for (size_t width = 1; width < runs; width *= 2)
        for (size_t i = 0; i + width < runs; i += 2 * width)
            std::inplace_merge(v.begin() + run[i], v.begin() + run[i + width],
                               v.begin() + run[std::min(i + 2 * width, runs)]);
}

// No output touches another, nor an input other than its own, nor the norm or the
// workspace, which no input touches either: both lists in the order of their addresses,
// walked side by side.
bool grads_apart(const std::vector<GradTensor> &t, const Bytes &norm, const Bytes &workspace, bool writes)
{
    std::vector<Bytes> in, out;
    in.reserve(t.size());
    out.reserve(t.size() + 2);
    for (const GradTensor &g : t) {
        const uintptr_t n = static_cast<uintptr_t>(g.n_flags >> kGradFlagBits);
        if (n == 0)
            continue;
        const uintptr_t src = reinterpret_cast<uintptr_t>(g.src), dst = reinterpret_cast<uintptr_t>(g.dst);
        const bool src16 = (g.n_flags & kGradSrcBf16) != 0, dst16 = (g.n_flags & kGradDstBf16) != 0;
        if (!(writes && src == dst && src16 == dst16))  // an input that is its own output is one list's alone
            in.push_back({src, src + n * (src16 ? 2 : 4)});
        if (writes)
            out.push_back({dst, dst + n * (dst16 ? 2 : 4)});
    }
    for (const Bytes &b : {norm, workspace})
        if (b.from != b.to)
            out.push_back(b);
    sort_bytes(in);
    sort_bytes(out);
    for (size_t i = 1; i < out.size(); ++i)
        if (out[i].from < out[i - 1].to)
            return false;
    // inputs may overlap each other: the furthest end so far stands for those that begin before an output
    size_t i = 0;
    uintptr_t end = 0;
    for (const Bytes &o : out) {
        for (; i < in.size() && in[i].from < o.to; ++i)
            end = in[i].to > end ? in[i].to : end;
        if (end > o.from)
            return false;
    }
    return true;
}

int clip(int64_t n, const void *const *grads, const int64_t *sizes, const int *dtypes, void *const *out,
         const int *out_dtypes, bool writes, float max_norm, float *norm, void *workspace, size_t ws_bytes,
         void *stream)
try {
    if (!norm || (writes && !(max_norm >= 0.0f)))
        return MXGEMM_ERR_ARG;
    std::vector<GradTensor> t;
    int st = read_grads(t, n, grads, sizes, dtypes, out, out_dtypes);
    if (st != MXGEMM_OK)
        return st;
    if (!aligned(norm, 4) || !aligned(workspace, 16))
        return MXGEMM_ERR_ALIGN;
    const size_t need = grad_workspace(n);
    if (need > 0 && (!workspace || ws_bytes < need))
        return MXGEMM_ERR_WORKSPACE;
    const uintptr_t a = reinterpret_cast<uintptr_t>(norm), w = reinterpret_cast<uintptr_t>(workspace);
    if (!grads_apart(t, {a, a + 4}, {w, w + need}, writes))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    st = ops_device(&sms);
    if (st != MXGEMM_OK)
        return st;
    double *partial = static_cast<double *>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return status_of(writes ? launch_clip_grads(t.data(), n, partial, max_norm, norm, sms, s)
                            : launch_grad_norm(t.data(), n, partial, norm, sms, s));
} catch (const std::bad_alloc &) {
    return MXGEMM_ERR_CUDA;
}

}  // namespace

extern "C" {

int mxgemm_embed(int in_dtype, const void *table, int64_t table_stride, int64_t vocab, int64_t K, const void *ids,
                 int id_bytes, int64_t tokens, float scale, int out_dtype, void *out, void *stream)
{
    if (!table || !ids || !out || !known_dtype(in_dtype) || !known_dtype(out_dtype) || !known_ids(id_bytes) ||
        !std::isfinite(scale))
        return MXGEMM_ERR_ARG;
    if (tokens < 1 || tokens > kMaxRows || vocab < 1 || vocab > kMaxRows || K < 32 || K % 32 != 0 || K > kMaxCols ||
        !rows_shape_ok(table, table_stride, vocab, K))
        return MXGEMM_ERR_SHAPE;
    const int64_t e = elem_bytes(in_dtype);
    if (!rows_align_ok(table, table_stride, vocab, e) || !aligned(ids, static_cast<unsigned>(id_bytes)) ||
        !aligned(out, 32))
        return MXGEMM_ERR_ALIGN;
    if (tokens * ((K + kWarpVals - 1) / kWarpVals) >= (1ll << 32) - 64)
        return MXGEMM_ERR_UNSUPPORTED;
    if (!outputs_apart({{dense(out, tokens, K * elem_bytes(out_dtype))}},
                       {{table, vocab, table_stride * e, K * e}, flat(ids, id_bytes * tokens)}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    const int st = ops_device(&sms);
    if (st != MXGEMM_OK)
        return st;
    EmbedParams p;
    p.table = bytes(table);
    p.table_stride = table_stride * e;
    p.vocab = vocab;
    p.K = K;
    p.ids = ids;
    p.ids64 = id_bytes == 8;
    p.tokens = tokens;
    p.scale = scale;
    p.out = static_cast<char *>(out);
    return status_of(launch_embed(p, in_dtype, out_dtype, sms, static_cast<cudaStream_t>(stream)));
}

// sizes that the gradient of the table takes: entries and their warps numbered in 32 bits
static bool embed_back_shape_ok(int64_t tokens, int64_t vocab, int64_t K)
{
    return tokens >= 1 && tokens <= kMaxRows && vocab >= 1 && vocab < kEmbedMaxVocab && K >= 32 && K % 32 == 0 &&
           K <= kMaxCols;
}
static bool embed_back_fits(int64_t tokens, int64_t vocab, int64_t K)
{
    const int64_t slices = (K + kWarpVals - 1) / kWarpVals;
    // warps of the sums; their blocks and, a row a warp at most, those that fill are below 2^31
    return slices < (1 << 16) && (tokens + 7) / 8 * slices < (1ll << 31);
}

size_t mxgemm_embed_backward_workspace_bytes(int64_t tokens, int64_t vocab, int64_t K)
{
    if (!embed_back_shape_ok(tokens, vocab, K) || !embed_back_fits(tokens, vocab, K))
        return 0;
    return embed_workspace(tokens, K).bytes;
}

int mxgemm_embed_backward(int in_dtype, const void *dy, int64_t dy_stride, const void *ids, int id_bytes,
                          int64_t tokens, int64_t vocab, int64_t K, float scale, const void *add, int out_dtype,
                          void *dtable, void *workspace, size_t ws_bytes, void *stream)
{
    if (!dy || !ids || !dtable || !known_dtype(in_dtype) || !known_dtype(out_dtype) || !known_ids(id_bytes) ||
        !std::isfinite(scale))
        return MXGEMM_ERR_ARG;
    if (!embed_back_shape_ok(tokens, vocab, K) || !rows_shape_ok(dy, dy_stride, tokens, K))
        return MXGEMM_ERR_SHAPE;
    const int64_t e = elem_bytes(in_dtype), row = K * elem_bytes(out_dtype);
    if (!rows_align_ok(dy, dy_stride, tokens, e) || !aligned(ids, static_cast<unsigned>(id_bytes)) ||
        !aligned(add, 32) || !aligned(dtable, 32) || !aligned(workspace, 32))
        return MXGEMM_ERR_ALIGN;
    if (!embed_back_fits(tokens, vocab, K))
        return MXGEMM_ERR_UNSUPPORTED;
    const size_t need = embed_workspace(tokens, K).bytes;
    if (need > 0 && (!workspace || ws_bytes < need))
        return MXGEMM_ERR_WORKSPACE;
    if (!outputs_apart({{dense(dtable, vocab, row), 0b1},
                        {flat(need > 0 ? workspace : nullptr, static_cast<int64_t>(need))}},
                       {dense(add, vocab, row),
                        {dy, tokens, dy_stride * e, K * e},
                        flat(ids, id_bytes * tokens)}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    const int st = ops_device(&sms, kEmbedGradient);
    if (st != MXGEMM_OK)
        return st;
    EmbedBackParams p = {};
    p.dy = bytes(dy);
    p.dy_stride = dy_stride * e;
    p.tokens = tokens;
    p.K = K;
    p.vocab = static_cast<uint32_t>(vocab);
    p.scale = scale;
    p.add = bytes(add);
    p.dtable = static_cast<char *>(dtable);
    return status_of(launch_embed_backward(p, ids, id_bytes == 8, static_cast<char *>(workspace), in_dtype, out_dtype,
                                           static_cast<cudaStream_t>(stream)));
}

int mxgemm_qk_norm_rope(int in_dtype, const void *x, int64_t x_token_stride, int64_t x_head_stride, int64_t tokens,
                        int64_t q_heads, int64_t k_heads, int64_t D, const void *q_weight, const void *k_weight,
                        int weight_dtype, float eps, const float *rope, int64_t rope_rows, int64_t rotary,
                        const void *positions, int position_bytes, uint32_t flags, void *y, int64_t y_token_stride,
                        int64_t y_head_stride, float *rstd, void *stream)
{
    const bool norm = q_weight || k_weight;
    if (!x || !y || (norm && ((q_heads > 0 && !q_weight) || (k_heads > 0 && !k_weight) || !(eps >= 0.0f))) ||
        (!norm && rstd))
        return MXGEMM_ERR_ARG;
    int st = check_heads(in_dtype, weight_dtype, norm, tokens, q_heads, k_heads, D, rope, rope_rows, rotary, positions,
                         position_bytes, flags);
    if (st != MXGEMM_OK)
        return st;
    const int64_t heads = q_heads + k_heads, e = elem_bytes(in_dtype);
    const Heads in = {x, x_token_stride, x_head_stride}, to = {y, y_token_stride, y_head_stride};
    if (!heads_shape_ok(in, tokens, heads, D) || !heads_shape_ok(to, tokens, heads, D))
        return MXGEMM_ERR_SHAPE;
    if (!heads_align_ok(in, tokens, heads, e) || !heads_align_ok(to, tokens, heads, e) || !aligned(q_weight, 32) ||
        !aligned(k_weight, 32) || !aligned(rstd, 4))
        return MXGEMM_ERR_ALIGN;
    const int64_t w = norm ? D * elem_bytes(weight_dtype) : 0;
    if (!outputs_apart({{heads_span(to, tokens, heads, D, e)}, {flat(rstd, 4 * tokens * heads)}},
                       {same_heads(in, to, tokens, heads) ? Span{} : heads_span(in, tokens, heads, D, e),
                        flat(q_weight, w),
                        flat(k_weight, w),
                        flat(rope, 4 * rope_rows * rotary),
                        flat(positions, position_bytes * tokens)}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    st = ops_device(&sms, kHeads);
    if (st != MXGEMM_OK)
        return st;
    HeadsParams p = {};
    set_heads(p, e, tokens, q_heads, k_heads, D, in, q_weight, k_weight, rope, rope_rows, rotary, positions,
              position_bytes);
    p.eps = eps;
    p.y = static_cast<char *>(y);
    p.y_token = y_token_stride * e;
    p.y_head = y_head_stride * e;
    p.rstd = rstd;
    return status_of(launch_heads(p, in_dtype, norm ? weight_dtype : 0, (flags & MXGEMM_ROPE_INTERLEAVED) != 0, sms,
                                  static_cast<cudaStream_t>(stream)));
}

size_t mxgemm_qk_norm_rope_backward_workspace_bytes(int64_t tokens, int64_t heads, int64_t D)
{
    if (tokens < 1 || tokens > kMaxRows || heads < 1 || heads > kMaxRows / tokens || D < 16 || D % 16 != 0 ||
        D > kHeadsMaxDim)
        return 0;
    return static_cast<size_t>(heads_back_blocks(tokens, static_cast<int>(heads), static_cast<int>(D)) * 2 * D) *
           sizeof(float);
}

int mxgemm_qk_norm_rope_backward(int in_dtype, const void *dy, int64_t dy_token_stride, int64_t dy_head_stride,
                                 const void *x, int64_t x_token_stride, int64_t x_head_stride, const float *rstd,
                                 int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t D, const void *q_weight,
                                 const void *k_weight, int weight_dtype, const float *rope, int64_t rope_rows,
                                 int64_t rotary, const void *positions, int position_bytes, uint32_t flags, void *dx,
                                 int64_t dx_token_stride, int64_t dx_head_stride, float *dq_weight, float *dk_weight,
                                 void *workspace, size_t ws_bytes, void *stream)
{
    const bool norm = q_weight || k_weight;
    if (!dy || !dx || (norm && ((q_heads > 0 && !q_weight) || (k_heads > 0 && !k_weight) || !x || !rstd)) ||
        (!norm && (rstd || dq_weight || dk_weight)))
        return MXGEMM_ERR_ARG;
    int st = check_heads(in_dtype, weight_dtype, norm, tokens, q_heads, k_heads, D, rope, rope_rows, rotary, positions,
                         position_bytes, flags);
    if (st != MXGEMM_OK)
        return st;
    const int64_t heads = q_heads + k_heads, e = elem_bytes(in_dtype);
    const Heads from = {dy, dy_token_stride, dy_head_stride}, to = {dx, dx_token_stride, dx_head_stride},
                in = {norm ? x : nullptr, x_token_stride, x_head_stride};
    if (!heads_shape_ok(from, tokens, heads, D) || !heads_shape_ok(to, tokens, heads, D) ||
        !heads_shape_ok(in, tokens, heads, D))
        return MXGEMM_ERR_SHAPE;
    if (!heads_align_ok(from, tokens, heads, e) || !heads_align_ok(to, tokens, heads, e) ||
        !heads_align_ok(in, tokens, heads, e) || !aligned(q_weight, 32) || !aligned(k_weight, 32) ||
        !aligned(rstd, 4) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned(workspace, 32))
        return MXGEMM_ERR_ALIGN;
    const size_t need = norm ? mxgemm_qk_norm_rope_backward_workspace_bytes(tokens, heads, D) : 0;
    if (need > 0 && (!workspace || ws_bytes < need))
        return MXGEMM_ERR_WORKSPACE;
    const int64_t w = norm ? D * elem_bytes(weight_dtype) : 0;
    if (!outputs_apart({{heads_span(to, tokens, heads, D, e)},
                        {flat(dq_weight, 4 * D)},
                        {flat(dk_weight, 4 * D)},
                        {flat(need > 0 ? workspace : nullptr, static_cast<int64_t>(need))}},
                       {same_heads(from, to, tokens, heads) ? Span{} : heads_span(from, tokens, heads, D, e),
                        same_heads(in, to, tokens, heads) ? Span{} : heads_span(in, tokens, heads, D, e),
                        flat(rstd, 4 * tokens * heads),
                        flat(q_weight, w),
                        flat(k_weight, w),
                        flat(rope, 4 * rope_rows * rotary),
                        flat(positions, position_bytes * tokens)}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    st = ops_device(&sms, kHeads);
    if (st != MXGEMM_OK)
        return st;
    const bool interleaved = (flags & MXGEMM_ROPE_INTERLEAVED) != 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!norm) {  // the rotation alone: the gradient goes back by the same angles
        HeadsParams p = {};
        set_heads(p, e, tokens, q_heads, k_heads, D, from, nullptr, nullptr, rope, rope_rows, rotary, positions,
                  position_bytes);
        p.inverse = true;
        p.y = static_cast<char *>(dx);
        p.y_token = dx_token_stride * e;
        p.y_head = dx_head_stride * e;
        return status_of(launch_heads(p, in_dtype, 0, interleaved, sms, s));
    }
    HeadsBackParams p = {};
    set_heads(p, e, tokens, q_heads, k_heads, D, in, q_weight, k_weight, rope, rope_rows, rotary, positions,
              position_bytes);
    p.dy = bytes(dy);
    p.dy_token = dy_token_stride * e;
    p.dy_head = dy_head_stride * e;
    p.rstd = rstd;
    p.dx = static_cast<char *>(dx);
    p.dx_token = dx_token_stride * e;
    p.dx_head = dx_head_stride * e;
    p.dq_weight = dq_weight;
    p.dk_weight = dk_weight;
    p.partial = static_cast<float *>(workspace);
    return status_of(launch_heads_backward(p, in_dtype, weight_dtype, interleaved, sms, s));
}

int mxgemm_logprobs(int in_dtype, const void *logits, int64_t stride, int64_t rows, int64_t V, float scale,
                    const void *targets, int id_bytes, float *logprob, float *entropy, float *stats, int64_t top,
                    int64_t *top_ids, float *top_logprobs, void *stream)
{
    if (!logits || !known_dtype(in_dtype) || !scale_ok(scale) ||
        (targets != nullptr) != (logprob != nullptr) || (targets && !known_ids(id_bytes)) ||
        (top != 0) != (top_ids != nullptr) || (top != 0) != (top_logprobs != nullptr) ||
        (!logprob && !entropy && !stats && top == 0))
        return MXGEMM_ERR_ARG;
    if (rows < 1 || rows > kMaxRows || V < 1 || V > kMaxCols || top < 0 || !logits_shape_ok(stride, rows, V))
        return MXGEMM_ERR_SHAPE;
    const int64_t e = elem_bytes(in_dtype);
    if (!aligned(logits, static_cast<unsigned>(e)) || (targets && !aligned(targets, static_cast<unsigned>(id_bytes))) ||
        !aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(stats, 8) || !aligned(top_ids, 8) ||
        !aligned(top_logprobs, 4))
        return MXGEMM_ERR_ALIGN;
    if (top > kLogprobsMaxTop || !logprobs_fits(rows, V))
        return MXGEMM_ERR_UNSUPPORTED;
    if (!outputs_apart({{flat(logprob, 4 * rows)},
                        {flat(entropy, 4 * rows)},
                        {flat(stats, 8 * rows)},
                        {flat(top_ids, 8 * rows * top)},
                        {flat(top_logprobs, 4 * rows * top)}},
                       {{logits, rows, stride * e, V * e}, flat(targets, id_bytes * rows)}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    const int st = ops_device(&sms);
    if (st != MXGEMM_OK)
        return st;
    LogprobsParams p;
    p.x = bytes(logits);
    p.stride = stride * e;
    p.rows = rows;
    p.V = V;
    p.scale = scale;
    p.targets = targets;
    p.targets64 = id_bytes == 8;
    p.logprob = logprob;
    p.entropy = entropy;
    p.stats = stats;
    p.top = static_cast<int>(top);
    p.top_ids = top_ids;
    p.top_logprobs = top_logprobs;
    return status_of(launch_logprobs(p, in_dtype, sms, static_cast<cudaStream_t>(stream)));
}

int mxgemm_logprobs_backward(int in_dtype, const void *logits, int64_t stride, int64_t rows, int64_t V, float scale,
                             const void *targets, int id_bytes, const float *stats, const float *dlogprob,
                             const float *entropy, const float *dentropy, void *dlogits, int64_t dlogits_stride,
                             void *stream)
{
    if (!logits || !stats || !dlogits || !known_dtype(in_dtype) || !scale_ok(scale) ||
        (targets != nullptr) != (dlogprob != nullptr) || (targets && !known_ids(id_bytes)) ||
        (dentropy && !entropy) || (!dlogprob && !dentropy))
        return MXGEMM_ERR_ARG;
    if (rows < 1 || rows > kMaxRows || V < 1 || V > kMaxCols || !logits_shape_ok(stride, rows, V) ||
        !logits_shape_ok(dlogits_stride, rows, V))
        return MXGEMM_ERR_SHAPE;
    const int64_t e = elem_bytes(in_dtype);
    if (!aligned(logits, static_cast<unsigned>(e)) || (targets && !aligned(targets, static_cast<unsigned>(id_bytes))) ||
        !aligned(stats, 8) || !aligned(dlogprob, 4) || !aligned(entropy, 4) || !aligned(dentropy, 4) ||
        !aligned(dlogits, static_cast<unsigned>(e)))
        return MXGEMM_ERR_ALIGN;
    if (!logprobs_fits(rows, V))
        return MXGEMM_ERR_UNSUPPORTED;
    const bool same = dlogits == logits && (rows == 1 || dlogits_stride == stride);
    if (!outputs_apart({{{dlogits, rows, dlogits_stride * e, V * e}}},
                       {same ? Span{} : Span{logits, rows, stride * e, V * e},
                        flat(targets, id_bytes * rows),
                        flat(stats, 8 * rows),
                        flat(dlogprob, 4 * rows),
                        flat(dentropy ? entropy : nullptr, 4 * rows),
                        flat(dentropy, 4 * rows)}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    const int st = ops_device(&sms);
    if (st != MXGEMM_OK)
        return st;
    LogprobsBackParams p;
    p.x = bytes(logits);
    p.stride = stride * e;
    p.rows = rows;
    p.V = V;
    p.scale = scale;
    p.targets = targets;
    p.targets64 = id_bytes == 8;
    p.stats = stats;
    p.dlogprob = dlogprob;
    p.entropy = entropy;
    p.dentropy = dentropy;
    p.dlogits = static_cast<char *>(dlogits);
    p.dlogits_stride = dlogits_stride * e;
    return status_of(launch_logprobs_backward(p, in_dtype, static_cast<cudaStream_t>(stream)));
}

size_t mxgemm_grad_workspace_bytes(int64_t n) { return n < 1 || n > (1 << 20) ? 0 : grad_workspace(n); }

int mxgemm_grad_norm(int64_t n, const void *const *grads, const int64_t *sizes, const int *dtypes, float *norm,
                     void *workspace, size_t ws_bytes, void *stream)
{
    return clip(n, grads, sizes, dtypes, nullptr, nullptr, false, 0.0f, norm, workspace, ws_bytes, stream);
}

int mxgemm_clip_grads(int64_t n, const void *const *grads, const int64_t *sizes, const int *dtypes, void *const *out,
                      const int *out_dtypes, float max_norm, float *norm, void *workspace, size_t ws_bytes,
                      void *stream)
{
    return clip(n, grads, sizes, dtypes, out, out_dtypes, true, max_norm, norm, workspace, ws_bytes, stream);
}

}  // extern "C"
