// ops.h -- internal interface of the row operators around the GEMM: RMS norm
// (norm.cu), gated activation (glu.cu), expert dispatch and combine (moe.cu).
// The launchers take arguments that the C ABI (ops.cu) has checked.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace mxg {

// Launch configuration of the row operators: programmatic stream serialization,
// so a kernel's CTAs may become resident while the preceding kernel drains; each
// kernel waits for it (griddepcontrol.wait) before its first access to memory.  One
// exception: the expert sort reads its ids before it waits for its own counting kernel,
// which lets it start only after a wait of its own.
inline cudaLaunchConfig_t row_launch(unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                                     cudaLaunchAttribute (&attr)[1])
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// An MX output: format kNoFmt (absent), kMxfp8 or kMxfp4, codes in dense rows.
struct MxOut {
    int fmt;
    int mode;         // kScaleBytes, kScaleWords or kScaleTiled
    uint8_t *codes;
    uint8_t *scales;
};

struct NormParams {
    const char *x, *residual;             // residual may be NULL
    int64_t x_stride, residual_stride;    // bytes from row to row
    const char *weight;
    int64_t rows, K;
    float eps;
    char *h, *y;                          // dense rows of the input type, or NULL
    float *rstd;                          // or NULL
    MxOut mx;
};
constexpr int64_t kNormMaxK = 32768;
cudaError_t launch_rmsnorm(const NormParams &p, int in_dtype, int weight_dtype, cudaStream_t s);

struct NormBackParams {
    const char *dy, *h, *dh;                       // dh may be NULL
    int64_t dy_stride, h_stride, dh_stride;        // bytes from row to row
    const float *rstd;
    const char *weight;
    int64_t rows, K;
    char *dx;                                      // dense rows
    float *dweight;
    float *partial;                                // [blocks][K]
};
// Blocks of the first pass at most (each leaves one row of partial sums; none where
// one launch does it all), on a part of at most kNormBackSms multiprocessors.
constexpr int kNormBackSms = 152;
int64_t norm_back_blocks(int64_t rows, int64_t K);
// Set the backward kernels' shared-memory opt-in on the current device; once per
// device, before the first launch.
cudaError_t prepare_norm();
cudaError_t launch_rmsnorm_backward(const NormBackParams &p, int in_dtype, int weight_dtype, int num_sms,
                                    cudaStream_t s);

constexpr int kActSilu = 1;
constexpr int kActGeluTanh = 2;

struct GluParams {
    const char *gate, *up;
    int64_t stride;                // bytes from row to row, of both
    int64_t rows, F;
    char *y;                       // dense rows, or NULL
    MxOut mx;
    uint8_t *kept_codes;           // rows x 2F MXFP8 codes (gate | up), or NULL
    uint8_t *kept_scales;          // rows x 2F/32, row-major
};
cudaError_t launch_glu(const GluParams &p, int act, int in_dtype, int num_sms, cudaStream_t s);

struct GluBackParams {
    const char *dy;
    int64_t dy_stride;             // bytes
    const char *gate, *up;         // NULL: from the kept codes
    int64_t stride;                // bytes
    const uint8_t *kept_codes, *kept_scales;
    int64_t rows, F;
    char *dgu;                     // dense rows of 2F values (dgate | dup), or NULL
    char *a;                       // dense rows of F values, or NULL
    MxOut mx;                      // of [dgate | dup], rows of 2F
};
cudaError_t launch_glu_backward(const GluBackParams &p, int act, int in_dtype, int num_sms, cudaStream_t s);

// Expert ids 0 .. groups - 1, as many as a grouped GEMM plan takes.
constexpr int kMaxSortGroups = 512;
// Blocks that share a sort, and the bytes of `counts` that it needs.
int64_t sort_tiles(int64_t slots, int64_t groups);
size_t sort_workspace(int64_t slots, int64_t groups);
cudaError_t launch_moe_sort(const void *ids, bool ids64, int64_t slots, int groups, int64_t *offsets,
                            int32_t *row_of_slot, int32_t *slot_of_row, int *counts, cudaStream_t s);

struct DispatchParams {
    const char *x;
    int64_t x_stride;              // bytes
    int64_t tokens, topk, K;
    const int32_t *row_of_slot;
    int fmt;                       // kMxfp8, kMxfp4 or kRowsBf16
    int mode;                      // kScaleBytes or kScaleWords
    uint8_t *rows;
    uint8_t *scales;
};
cudaError_t launch_moe_dispatch(const DispatchParams &p, int in_dtype, int num_sms, cudaStream_t s);

struct CombineParams {
    const char *y;
    int64_t y_stride;              // bytes
    int64_t tokens, topk, N;
    const int32_t *row_of_slot;
    const float *weights;          // tokens x topk, or NULL (all 1)
    const char *add;               // or NULL
    int64_t add_stride;            // bytes
    char *out;                     // dense rows
};
cudaError_t launch_moe_combine(const CombineParams &p, int in_dtype, int num_sms, cudaStream_t s);

struct CombineBackParams {
    const char *dout, *y;
    int64_t dout_stride, y_stride; // bytes
    int64_t tokens, topk, N;
    const int32_t *row_of_slot;
    const float *weights;
    char *dy;                      // dense rows
    float *dweights;
};
cudaError_t launch_moe_combine_backward(const CombineBackParams &p, int in_dtype, int num_sms, cudaStream_t s);

}  // namespace mxg
