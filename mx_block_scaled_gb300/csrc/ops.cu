// ops.cu -- C ABI of the row operators around the GEMM (RMS norm, gated
// activation, expert sort / dispatch / combine): argument checks and launches.
#include "ops.h"

#include <initializer_list>
#include <mutex>

#include "mx_block.cuh"
#include "mxgemm.h"

namespace {

constexpr int kMaxDevices = 64;

struct OpsDevice {
    bool ready = false;
    bool is_sm103 = false;
    int num_sms = 0;
};
OpsDevice g_ops_dev[kMaxDevices];
std::mutex g_ops_mutex;

// The current device's SM count; prepares it on first use.
int ops_device(int *num_sms)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return MXGEMM_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_ops_mutex);
    OpsDevice &d = g_ops_dev[dev];
    if (!d.ready) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return MXGEMM_ERR_CUDA;
        d.is_sm103 = major == 10 && minor == 3;
        if (d.is_sm103 && mxg::prepare_norm() != cudaSuccess)
            return MXGEMM_ERR_CUDA;
        d.ready = true;
    }
    *num_sms = d.num_sms;
    return d.is_sm103 ? MXGEMM_OK : MXGEMM_ERR_ARCH;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? MXGEMM_OK : MXGEMM_ERR_CUDA; }

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int64_t kMaxRows = (1ll << 31) - 1;
constexpr int64_t kMaxCols = 1ll << 30;

bool known_dtype(int d) { return d == MXGEMM_IN_F32 || d == MXGEMM_IN_BF16; }
int64_t elem_bytes(int d) { return d == MXGEMM_IN_BF16 ? 2 : 4; }
const char *bytes(const void *p) { return static_cast<const char *>(p); }

// A strided input matrix: NULL passes; rows start on 32-byte boundaries and do
// not overlap (a stride of at least the row, or a single row).
bool rows_shape_ok(const void *p, int64_t stride, int64_t rows, int64_t cols)
{
    return p == nullptr || rows == 1 || (stride >= cols && stride <= (1ll << 40));
}
bool rows_align_ok(const void *p, int64_t stride, int64_t rows, int64_t elem)
{
    return p == nullptr || (aligned(p, 32) && (rows == 1 || stride * elem % 32 == 0));
}

// Bytes of a matrix, from its first to its last; p NULL for one that there is not.
struct Span {
    const void *p;
    int64_t rows, stride, row;
};
Span dense(const void *p, int64_t rows, int64_t row) { return {p, rows, row, row}; }
Span flat(const void *p, int64_t n) { return {p, 1, n, n}; }

bool apart(const Span &a, const Span &b)
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
bool outputs_apart(std::initializer_list<Output> outs, std::initializer_list<Span> ins)
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

// Bytes of a row of n MX codes.
int64_t code_bytes(int fmt, int64_t n) { return fmt == MXGEMM_FMT_MXFP4_E2M1 ? n / 2 : n; }

// Bytes of the scales of [rows, K].
int64_t scale_bytes(uint32_t flags, int64_t rows, int64_t K)
{
    return ((flags & MXGEMM_QUANT_SF_TILED) ? (rows + 127) / 128 * 128 : rows) * (K / 32);
}

// The MX output of a call: fmt 0 has neither codes nor scales.
int check_mx(int fmt, const void *codes, const uint8_t *scales, uint32_t flags, int64_t K)
{
    if (flags & ~MXGEMM_QUANT_SF_TILED)
        return MXGEMM_ERR_ARG;
    if (fmt == 0)
        return codes || scales || flags ? MXGEMM_ERR_ARG : MXGEMM_OK;
    if ((fmt != MXGEMM_FMT_MXFP8_E4M3 && fmt != MXGEMM_FMT_MXFP4_E2M1) || !codes || !scales)
        return MXGEMM_ERR_ARG;
    if ((flags & MXGEMM_QUANT_SF_TILED) && K % 128 != 0)
        return MXGEMM_ERR_SHAPE;
    return aligned(codes, 16) && aligned(scales, 16) ? MXGEMM_OK : MXGEMM_ERR_ALIGN;
}

mxg::MxOut make_mx(int fmt, void *codes, uint8_t *scales, uint32_t flags, int64_t K)
{
    mxg::MxOut m;
    m.fmt = fmt;
    m.mode = (flags & MXGEMM_QUANT_SF_TILED) ? mxg::kScaleTiled : K % 128 == 0 ? mxg::kScaleWords : mxg::kScaleBytes;
    m.codes = static_cast<uint8_t *>(codes);
    m.scales = scales;
    return m;
}

}  // namespace

extern "C" {

int mxgemm_rmsnorm(int in_dtype, const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                   const void *weight, int weight_dtype, float eps, int64_t rows, int64_t K, void *h, void *y, int fmt,
                   void *codes, uint8_t *scales, float *rstd, uint32_t flags, void *stream)
{
    if (!x || !weight || !known_dtype(in_dtype) || !known_dtype(weight_dtype) || !(eps >= 0.0f))
        return MXGEMM_ERR_ARG;
    if (!h && !y && fmt == 0 && !rstd)
        return MXGEMM_ERR_ARG;
    if (rows < 1 || rows > kMaxRows || K < 32 || K % 32 != 0 || K > kMaxCols ||
        !rows_shape_ok(x, x_stride, rows, K) || !rows_shape_ok(residual, residual_stride, rows, K))
        return MXGEMM_ERR_SHAPE;
    int st = check_mx(fmt, codes, scales, flags, K);
    if (st != MXGEMM_OK)
        return st;
    const int64_t e = elem_bytes(in_dtype);
    if (!rows_align_ok(x, x_stride, rows, e) || !rows_align_ok(residual, residual_stride, rows, e) ||
        !aligned(weight, 32) || !aligned(h, 32) || !aligned(y, 32) || !aligned(rstd, 4))
        return MXGEMM_ERR_ALIGN;
    if (K > mxg::kNormMaxK)
        return MXGEMM_ERR_UNSUPPORTED;
    const int64_t row = K * e;
    if (!outputs_apart({{dense(h, rows, row), 0b11},
                        {dense(y, rows, row), 0b11},
                        {dense(codes, rows, code_bytes(fmt, K))},
                        {flat(scales, scale_bytes(flags, rows, K))},
                        {flat(rstd, 4 * rows)}},
                       {{x, rows, x_stride * e, row},
                        {residual, rows, residual_stride * e, row},
                        flat(weight, K * elem_bytes(weight_dtype))}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    st = ops_device(&sms);
    if (st != MXGEMM_OK)
        return st;
    mxg::NormParams p;
    p.x = bytes(x);
    p.x_stride = x_stride * e;
    p.residual = bytes(residual);
    p.residual_stride = residual_stride * e;
    p.weight = bytes(weight);
    p.rows = rows;
    p.K = K;
    p.eps = eps;
    p.h = static_cast<char *>(h);
    p.y = static_cast<char *>(y);
    p.rstd = rstd;
    p.mx = make_mx(fmt, codes, scales, flags, K);
    return status_of(mxg::launch_rmsnorm(p, in_dtype, weight_dtype, static_cast<cudaStream_t>(stream)));
}

size_t mxgemm_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t K)
{
    if (rows < 1 || rows > kMaxRows || K < 32 || K % 32 != 0 || K > mxg::kNormMaxK)
        return 0;
    return static_cast<size_t>(mxg::norm_back_blocks(rows, K) * K) * sizeof(float);
}

int mxgemm_rmsnorm_backward(int in_dtype, const void *dy, int64_t dy_stride, const void *h, int64_t h_stride,
                            const float *rstd, const void *weight, int weight_dtype, const void *dh, int64_t dh_stride,
                            int64_t rows, int64_t K, void *dx, float *dweight, void *workspace, size_t ws_bytes,
                            void *stream)
{
    if (!dy || !h || !rstd || !weight || !dx || !dweight || !known_dtype(in_dtype) || !known_dtype(weight_dtype))
        return MXGEMM_ERR_ARG;
    if (rows < 1 || rows > kMaxRows || K < 32 || K % 32 != 0 || K > kMaxCols ||
        !rows_shape_ok(dy, dy_stride, rows, K) || !rows_shape_ok(h, h_stride, rows, K) ||
        !rows_shape_ok(dh, dh_stride, rows, K))
        return MXGEMM_ERR_SHAPE;
    const int64_t e = elem_bytes(in_dtype);
    if (!rows_align_ok(dy, dy_stride, rows, e) || !rows_align_ok(h, h_stride, rows, e) ||
        !rows_align_ok(dh, dh_stride, rows, e) || !aligned(weight, 32) || !aligned(dx, 32) || !aligned(dweight, 32) ||
        !aligned(rstd, 4) || !aligned(workspace, 32))
        return MXGEMM_ERR_ALIGN;
    if (K > mxg::kNormMaxK)
        return MXGEMM_ERR_UNSUPPORTED;
    const size_t need = mxgemm_rmsnorm_backward_workspace_bytes(rows, K);
    if (need > 0 && (!workspace || ws_bytes < need))
        return MXGEMM_ERR_WORKSPACE;
    const int64_t row = K * e;
    if (!outputs_apart({{dense(dx, rows, row), 0b100},
                        {flat(dweight, 4 * K)},
                        {flat(need > 0 ? workspace : nullptr, static_cast<int64_t>(need))}},
                       {{dy, rows, dy_stride * e, row},
                        {h, rows, h_stride * e, row},
                        {dh, rows, dh_stride * e, row},
                        flat(rstd, 4 * rows),
                        flat(weight, K * elem_bytes(weight_dtype))}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    const int st = ops_device(&sms);
    if (st != MXGEMM_OK)
        return st;
    mxg::NormBackParams p;
    p.dy = bytes(dy);
    p.dy_stride = dy_stride * e;
    p.h = bytes(h);
    p.h_stride = h_stride * e;
    p.dh = bytes(dh);
    p.dh_stride = dh_stride * e;
    p.rstd = rstd;
    p.weight = bytes(weight);
    p.rows = rows;
    p.K = K;
    p.dx = static_cast<char *>(dx);
    p.dweight = dweight;
    p.partial = static_cast<float *>(workspace);
    return status_of(mxg::launch_rmsnorm_backward(p, in_dtype, weight_dtype, sms, static_cast<cudaStream_t>(stream)));
}

int mxgemm_glu(int act, int in_dtype, const void *gate, const void *up, int64_t stride, int64_t rows, int64_t F,
               void *y, int fmt, void *codes, uint8_t *scales, uint32_t flags, void *kept_codes, uint8_t *kept_scales,
               void *stream)
{
    if (!gate || !up || !known_dtype(in_dtype) || (act != MXGEMM_ACT_SILU && act != MXGEMM_ACT_GELU_TANH) ||
        (kept_codes == nullptr) != (kept_scales == nullptr))
        return MXGEMM_ERR_ARG;
    if (!y && fmt == 0 && !kept_codes)
        return MXGEMM_ERR_ARG;
    if (rows < 1 || rows > kMaxRows || F < 32 || F % 32 != 0 || F > kMaxCols || !rows_shape_ok(gate, stride, rows, F))
        return MXGEMM_ERR_SHAPE;
    int st = check_mx(fmt, codes, scales, flags, F);
    if (st != MXGEMM_OK)
        return st;
    const int64_t e = elem_bytes(in_dtype);
    if (!rows_align_ok(gate, stride, rows, e) || !aligned(up, 32) || !aligned(y, 32) || !aligned(kept_codes, 16) ||
        !aligned(kept_scales, 16))
        return MXGEMM_ERR_ALIGN;
    const int64_t row = F * e;
    if (!outputs_apart({{dense(y, rows, row), 0b11},
                        {dense(codes, rows, code_bytes(fmt, F))},
                        {flat(scales, scale_bytes(flags, rows, F))},
                        {dense(kept_codes, rows, 2 * F)},
                        {flat(kept_scales, scale_bytes(0, rows, 2 * F))}},
                       {{gate, rows, stride * e, row}, {up, rows, stride * e, row}}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    st = ops_device(&sms);
    if (st != MXGEMM_OK)
        return st;
    mxg::GluParams p;
    p.gate = bytes(gate);
    p.up = bytes(up);
    p.stride = stride * e;
    p.rows = rows;
    p.F = F;
    p.y = static_cast<char *>(y);
    p.mx = make_mx(fmt, codes, scales, flags, F);
    p.kept_codes = static_cast<uint8_t *>(kept_codes);
    p.kept_scales = kept_scales;
    return status_of(mxg::launch_glu(p, act, in_dtype, sms, static_cast<cudaStream_t>(stream)));
}

int mxgemm_glu_backward(int act, int in_dtype, const void *dy, int64_t dy_stride, const void *gate, const void *up,
                        int64_t stride, const void *kept_codes, const uint8_t *kept_scales, int64_t rows, int64_t F,
                        void *dgu, int fmt, void *codes, uint8_t *scales, uint32_t flags, void *a, void *stream)
{
    if (!dy || !known_dtype(in_dtype) || (act != MXGEMM_ACT_SILU && act != MXGEMM_ACT_GELU_TANH))
        return MXGEMM_ERR_ARG;
    // the inputs come either as they were or as the forward's checkpoint
    const bool kept = kept_codes != nullptr;
    if (kept != (kept_scales != nullptr) || (gate != nullptr) != (up != nullptr) || kept == (gate != nullptr))
        return MXGEMM_ERR_ARG;
    if (!dgu && fmt == 0 && !a)
        return MXGEMM_ERR_ARG;
    if (rows < 1 || rows > kMaxRows || F < 32 || F % 32 != 0 || F > kMaxCols / 2 ||
        !rows_shape_ok(dy, dy_stride, rows, F) || !rows_shape_ok(gate, stride, rows, F))
        return MXGEMM_ERR_SHAPE;
    int st = check_mx(fmt, codes, scales, flags, 2 * F);
    if (st != MXGEMM_OK)
        return st;
    const int64_t e = elem_bytes(in_dtype);
    if (!rows_align_ok(dy, dy_stride, rows, e) || !rows_align_ok(gate, stride, rows, e) || !aligned(up, 32) ||
        !aligned(kept_codes, 16) || !aligned(kept_scales, 16) || !aligned(dgu, 32) || !aligned(a, 32))
        return MXGEMM_ERR_ALIGN;
    const int64_t row = F * e;
    // dgu may be the [rows, 2F] matrix that gate and up are the halves of: one input then
    const bool halves = dgu && dgu == gate && up == bytes(gate) + row && (rows == 1 || stride == 2 * F);
    if (!outputs_apart({{dense(dgu, rows, 2 * row), 0b10},
                        {dense(codes, rows, code_bytes(fmt, 2 * F))},
                        {flat(scales, scale_bytes(flags, rows, 2 * F))},
                        {dense(a, rows, row), 0b111}},
                       {{dy, rows, dy_stride * e, row},
                        halves ? dense(gate, rows, 2 * row) : Span{gate, rows, stride * e, row},
                        {halves ? nullptr : up, rows, stride * e, row},
                        dense(kept_codes, rows, 2 * F),
                        flat(kept_scales, scale_bytes(0, rows, 2 * F))}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    st = ops_device(&sms);
    if (st != MXGEMM_OK)
        return st;
    mxg::GluBackParams p;
    p.dy = bytes(dy);
    p.dy_stride = dy_stride * e;
    p.gate = bytes(gate);
    p.up = bytes(up);
    p.stride = stride * e;
    p.kept_codes = static_cast<const uint8_t *>(kept_codes);
    p.kept_scales = kept_scales;
    p.rows = rows;
    p.F = F;
    p.dgu = static_cast<char *>(dgu);
    p.a = static_cast<char *>(a);
    p.mx = make_mx(fmt, codes, scales, flags, 2 * F);
    return status_of(mxg::launch_glu_backward(p, act, in_dtype, sms, static_cast<cudaStream_t>(stream)));
}

size_t mxgemm_moe_sort_workspace_bytes(int64_t slots, int64_t groups)
{
    if (slots < 1 || slots > kMaxRows || groups < 1 || groups > mxg::kMaxSortGroups)
        return 0;
    return mxg::sort_workspace(slots, groups);
}

int mxgemm_moe_sort(const void *expert_ids, int id_bytes, int64_t slots, int64_t groups, int64_t *offsets,
                    int32_t *row_of_slot, int32_t *slot_of_row, void *workspace, size_t ws_bytes, void *stream)
{
    if (!expert_ids || !offsets || !row_of_slot || (id_bytes != 4 && id_bytes != 8))
        return MXGEMM_ERR_ARG;
    if (slots < 1 || slots > kMaxRows || groups < 1 || groups > mxg::kMaxSortGroups)
        return MXGEMM_ERR_SHAPE;
    if (!aligned(expert_ids, static_cast<unsigned>(id_bytes)) || !aligned(offsets, 8) || !aligned(row_of_slot, 4) ||
        !aligned(slot_of_row, 4) || !aligned(workspace, 16))
        return MXGEMM_ERR_ALIGN;
    const size_t need = mxgemm_moe_sort_workspace_bytes(slots, groups);
    if (need > 0 && (!workspace || ws_bytes < need))
        return MXGEMM_ERR_WORKSPACE;
    if (!outputs_apart({{flat(offsets, 8 * (groups + 1))},
                        {flat(row_of_slot, 4 * slots)},
                        {flat(slot_of_row, 4 * slots)},
                        {flat(need > 0 ? workspace : nullptr, static_cast<int64_t>(need))}},
                       {flat(expert_ids, id_bytes * slots)}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    const int st = ops_device(&sms);
    if (st != MXGEMM_OK)
        return st;
    return status_of(mxg::launch_moe_sort(expert_ids, id_bytes == 8, slots, static_cast<int>(groups), offsets,
                                          row_of_slot, slot_of_row, static_cast<int *>(workspace),
                                          static_cast<cudaStream_t>(stream)));
}

// tokens x topk slots fit the sort's 32-bit rows, and a token's slots a 32-bit count with room to step past it
static bool slots_ok(int64_t tokens, int64_t topk)
{
    return tokens >= 1 && topk >= 1 && topk <= (1 << 20) && tokens <= kMaxRows / topk;
}

// one warp for every 512 values of a token, numbered in 32 bits
static bool warps_ok(int64_t tokens, int64_t cols) { return tokens * ((cols + 511) / 512) < (1ll << 32) - 64; }

int mxgemm_moe_dispatch(int in_dtype, const void *x, int64_t x_stride, int64_t tokens, int64_t topk, int64_t K,
                        const int32_t *row_of_slot, int fmt, void *rows, uint8_t *scales, void *stream)
{
    if (!x || !row_of_slot || !rows || !known_dtype(in_dtype))
        return MXGEMM_ERR_ARG;
    const bool plain = fmt == MXGEMM_FMT_BF16;
    if ((!plain && fmt != MXGEMM_FMT_MXFP8_E4M3 && fmt != MXGEMM_FMT_MXFP4_E2M1) || plain == (scales != nullptr))
        return MXGEMM_ERR_ARG;
    if (!slots_ok(tokens, topk) || K < 32 || K % 32 != 0 || K > kMaxCols || !rows_shape_ok(x, x_stride, tokens, K))
        return MXGEMM_ERR_SHAPE;
    const int64_t e = elem_bytes(in_dtype);
    if (!rows_align_ok(x, x_stride, tokens, e) || !aligned(row_of_slot, 4) || !aligned(rows, plain ? 32 : 16) ||
        !aligned(scales, 16))
        return MXGEMM_ERR_ALIGN;
    if (!warps_ok(tokens, K))
        return MXGEMM_ERR_UNSUPPORTED;
    const int64_t slots = tokens * topk;
    if (!outputs_apart({{dense(rows, slots, plain ? 2 * K : code_bytes(fmt, K))}, {flat(scales, scale_bytes(0, slots, K))}},
                       {{x, tokens, x_stride * e, K * e}, flat(row_of_slot, 4 * slots)}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    const int st = ops_device(&sms);
    if (st != MXGEMM_OK)
        return st;
    mxg::DispatchParams p;
    p.x = bytes(x);
    p.x_stride = x_stride * e;
    p.tokens = tokens;
    p.topk = topk;
    p.K = K;
    p.row_of_slot = row_of_slot;
    p.fmt = fmt;
    p.mode = K % 128 == 0 ? mxg::kScaleWords : mxg::kScaleBytes;
    p.rows = static_cast<uint8_t *>(rows);
    p.scales = scales;
    return status_of(mxg::launch_moe_dispatch(p, in_dtype, sms, static_cast<cudaStream_t>(stream)));
}

int mxgemm_moe_combine(int in_dtype, const void *y, int64_t y_stride, int64_t tokens, int64_t topk, int64_t N,
                       const int32_t *row_of_slot, const float *weights, const void *add, int64_t add_stride,
                       void *out, void *stream)
{
    if (!y || !row_of_slot || !out || !known_dtype(in_dtype))
        return MXGEMM_ERR_ARG;
    if (!slots_ok(tokens, topk) || N < 32 || N % 32 != 0 || N > kMaxCols ||
        !rows_shape_ok(y, y_stride, tokens * topk, N) || !rows_shape_ok(add, add_stride, tokens, N))
        return MXGEMM_ERR_SHAPE;
    const int64_t e = elem_bytes(in_dtype);
    if (!rows_align_ok(y, y_stride, tokens * topk, e) || !rows_align_ok(add, add_stride, tokens, e) ||
        !aligned(row_of_slot, 4) || !aligned(weights, 4) || !aligned(out, 32))
        return MXGEMM_ERR_ALIGN;
    if (!warps_ok(tokens, N))
        return MXGEMM_ERR_UNSUPPORTED;
    const int64_t row = N * e, slots = tokens * topk;
    if (!outputs_apart({{dense(out, tokens, row), 0b10}},
                       {{y, slots, y_stride * e, row},
                        {add, tokens, add_stride * e, row},
                        flat(row_of_slot, 4 * slots),
                        flat(weights, 4 * slots)}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    const int st = ops_device(&sms);
    if (st != MXGEMM_OK)
        return st;
    mxg::CombineParams p;
    p.y = bytes(y);
    p.y_stride = y_stride * e;
    p.tokens = tokens;
    p.topk = topk;
    p.N = N;
    p.row_of_slot = row_of_slot;
    p.weights = weights;
    p.add = bytes(add);
    p.add_stride = add_stride * e;
    p.out = static_cast<char *>(out);
    return status_of(mxg::launch_moe_combine(p, in_dtype, sms, static_cast<cudaStream_t>(stream)));
}

int mxgemm_moe_combine_backward(int in_dtype, const void *dout, int64_t dout_stride, const void *y, int64_t y_stride,
                                int64_t tokens, int64_t topk, int64_t N, const int32_t *row_of_slot,
                                const float *weights, void *dy, float *dweights, void *stream)
{
    if (!dout || !y || !row_of_slot || !weights || !dy || !dweights || !known_dtype(in_dtype))
        return MXGEMM_ERR_ARG;
    if (!slots_ok(tokens, topk) || N < 32 || N % 32 != 0 || N > kMaxCols ||
        !rows_shape_ok(y, y_stride, tokens * topk, N) || !rows_shape_ok(dout, dout_stride, tokens, N))
        return MXGEMM_ERR_SHAPE;
    const int64_t e = elem_bytes(in_dtype);
    if (!rows_align_ok(y, y_stride, tokens * topk, e) || !rows_align_ok(dout, dout_stride, tokens, e) ||
        !aligned(row_of_slot, 4) || !aligned(weights, 4) || !aligned(dy, 32) || !aligned(dweights, 4))
        return MXGEMM_ERR_ALIGN;
    const int64_t row = N * e, slots = tokens * topk;
    if (!outputs_apart({{dense(dy, slots, row), 0b10}, {flat(dweights, 4 * slots), 0b1000}},
                       {{dout, tokens, dout_stride * e, row},
                        {y, slots, y_stride * e, row},
                        flat(row_of_slot, 4 * slots),
                        flat(weights, 4 * slots)}))
        return MXGEMM_ERR_ARG;
    int sms = 0;
    const int st = ops_device(&sms);
    if (st != MXGEMM_OK)
        return st;
    mxg::CombineBackParams p;
    p.dout = bytes(dout);
    p.dout_stride = dout_stride * e;
    p.y = bytes(y);
    p.y_stride = y_stride * e;
    p.tokens = tokens;
    p.topk = topk;
    p.N = N;
    p.row_of_slot = row_of_slot;
    p.weights = weights;
    p.dy = static_cast<char *>(dy);
    p.dweights = dweights;
    return status_of(mxg::launch_moe_combine_backward(p, in_dtype, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
