// ops.h -- internal interface of the row operators around the GEMM: RMS norm
// (norm.cu), gated activation (glu.cu), expert dispatch and combine (moe.cu); and
// of those at a model's ends and between its products: embedding (embed.cu), norm
// and rotation of heads (heads.cu), log probabilities (logprobs.cu), gradient norm
// and clipping (clip.cu).
// The launchers take arguments that the C ABI (ops.cu, ops_model.cu) has checked.
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

struct EmbedParams {
    const char *table;
    int64_t table_stride;          // bytes
    int64_t vocab, K;
    const void *ids;
    bool ids64;
    int64_t tokens;
    float scale;
    char *out;                     // dense rows
};
cudaError_t launch_embed(const EmbedParams &p, int in_dtype, int out_dtype, int num_sms, cudaStream_t s);

// The sort of a gradient's ids: passes of at most kEmbedDigitBits bits, a cluster of
// at most kEmbedSortTiles blocks.
constexpr int kEmbedDigitBits = 10;
constexpr int kEmbedSortTiles = 16;
constexpr int64_t kEmbedMaxVocab = 1ll << 30;
struct EmbedSortParams {
    const void *ids;
    bool ids64;
    int64_t tokens;
    uint32_t vocab;
    int bits, passes;              // passes 0: few tokens, sorted by counting
    int64_t run;                   // entries of a warp, a multiple of 32
    uint2 *entries0, *entries1;    // (id, token): the first pass writes entries0, the second entries1, and so on
    int *counts;                   // [blocks][2^kEmbedDigitBits]
};

struct EmbedBackParams {
    const char *dy;
    int64_t dy_stride;             // bytes
    int64_t tokens, K;
    uint32_t vocab;
    float scale;
    const char *add;               // dense rows of the gradient's type, or NULL; dtable itself: only rows that occur
    char *dtable;                  // dense rows
    const uint2 *entries;          // (id, token) sorted; this and the sums of parts are the launcher's
    float *partial;
};
struct EmbedWorkspace {
    int64_t entries[2], partial;   // bytes from the workspace's start
    size_t bytes;
};
EmbedWorkspace embed_workspace(int64_t tokens, int64_t K);
// Set the sort's shared-memory and cluster opt-in on the current device.
cudaError_t prepare_embed();
cudaError_t launch_embed_backward(EmbedBackParams p, const void *ids, bool ids64, char *workspace, int in_dtype,
                                  int out_dtype, cudaStream_t s);

// What the passes over heads have in common; strides in bytes.
struct HeadsCommon {
    int64_t tokens;
    int heads, q_heads, D, rotary;
    const char *q_weight, *k_weight;
    const float *rope;             // rope_rows x rotary (cos | sin), or NULL
    int64_t rope_rows;
    const void *positions;
    bool positions64;
    const char *x;
    int64_t x_token, x_head;
};
struct HeadsParams : HeadsCommon {
    float eps;
    bool inverse;                  // rotate by minus the angles
    char *y;
    int64_t y_token, y_head;
    float *rstd;                   // tokens x heads, or NULL
};
constexpr int kHeadsMaxDim = 512;
// weight_dtype 0: no norm
cudaError_t launch_heads(const HeadsParams &p, int in_dtype, int weight_dtype, bool interleaved, int num_sms,
                         cudaStream_t s);

struct HeadsBackParams : HeadsCommon {
    const char *dy;
    int64_t dy_token, dy_head;
    const float *rstd;
    char *dx;
    int64_t dx_token, dx_head;
    float *dq_weight, *dk_weight;  // either may be NULL
    float *partial;                // [blocks][2][D]
};
// Blocks that leave partial sums, at most, on a part of at most kHeadsBackSms multiprocessors (none for few tokens).
constexpr int kHeadsBackSms = 152;
constexpr int kHeadsBackPerSm = 3;
int64_t heads_back_blocks(int64_t tokens, int heads, int D);
// Set the kernels' shared-memory opt-in on the current device.
cudaError_t prepare_heads();
cudaError_t launch_heads_backward(const HeadsBackParams &p, int in_dtype, int weight_dtype, bool interleaved,
                                  int num_sms, cudaStream_t s);

struct LogprobsParams {
    const char *x;
    int64_t stride;                // bytes
    int64_t rows, V;
    float scale;
    const void *targets;           // or NULL
    bool targets64;
    float *logprob, *entropy, *stats;  // each or NULL; stats is rows x 2
    int top;
    int64_t *top_ids;
    float *top_logprobs;
};
constexpr int kLogprobsMaxTop = 32;
constexpr int kLogprobsCluster = 8;
bool logprobs_fits(int64_t rows, int64_t V);
cudaError_t launch_logprobs(const LogprobsParams &p, int in_dtype, int num_sms, cudaStream_t s);

struct LogprobsBackParams {
    const char *x;
    int64_t stride;                // bytes
    int64_t rows, V;
    float scale;
    const void *targets;
    bool targets64;
    const float *stats, *dlogprob, *entropy, *dentropy;  // dlogprob, or entropy and dentropy, may be NULL
    char *dlogits;
    int64_t dlogits_stride;        // bytes
};
cudaError_t launch_logprobs_backward(const LogprobsBackParams &p, int in_dtype, cudaStream_t s);

// Vector: the tensor starts on a 32-byte boundary.
constexpr uint32_t kGradSrcBf16 = 1, kGradDstBf16 = 2, kGradSrcVector = 4, kGradDstVector = 8;
constexpr int kGradFlagBits = 4;
struct GradTensor {
    const void *src;
    void *dst;
    int64_t n_flags;               // elements << kGradFlagBits, and the flags above
};
// Blocks of a launch (each leaves one partial sum) are on at most kGradSms multiprocessors.
constexpr int kGradSms = 152;
size_t grad_workspace(int64_t n);
bool grads_fit(const GradTensor *tensors, int64_t n);
cudaError_t launch_grad_norm(const GradTensor *tensors, int64_t n, double *partial, float *norm, int num_sms,
                             cudaStream_t s);
cudaError_t launch_clip_grads(const GradTensor *tensors, int64_t n, double *partial, float max_norm, float *norm,
                              int num_sms, cudaStream_t s);

}  // namespace mxg
