// rowops_py.cpp -- Python module _rowops: checks and marshalling of the row
// operators' tensors (binding.py has the public functions).
//
// A decode step calls these operators on a few rows, where a kernel takes 2 us: read
// through Python attributes and ctypes, a call's dozen tensors cost the host 7 to 13 us.
// Here a tensor's type, shape, strides and address are read from the tensor itself.
// The module has no arithmetic and calls the C ABI by the addresses that binding.py
// passes to bind(), so that it serves the release and the debug library alike.
//
// Every function returns a tuple of its outputs, or the int status of a call that the
// library refused; a tensor that does not fit raises ValueError before the call.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>
#include <stdexcept>
#include <string>
#include <vector>

#include "mxgemm.h"

namespace {

struct Entries {
    decltype(&mxgemm_rmsnorm) rmsnorm;
    decltype(&mxgemm_rmsnorm_backward_workspace_bytes) rmsnorm_backward_workspace_bytes;
    decltype(&mxgemm_rmsnorm_backward) rmsnorm_backward;
    decltype(&mxgemm_glu) glu;
    decltype(&mxgemm_glu_backward) glu_backward;
    decltype(&mxgemm_moe_sort_workspace_bytes) moe_sort_workspace_bytes;
    decltype(&mxgemm_moe_sort) moe_sort;
    decltype(&mxgemm_moe_dispatch) moe_dispatch;
    decltype(&mxgemm_moe_combine) moe_combine;
    decltype(&mxgemm_moe_combine_backward) moe_combine_backward;
    decltype(&mxgemm_sf_bytes) sf_bytes;
    decltype(&mxgemm_embed) embed;
    decltype(&mxgemm_embed_backward_workspace_bytes) embed_backward_workspace_bytes;
    decltype(&mxgemm_embed_backward) embed_backward;
    decltype(&mxgemm_qk_norm_rope) qk_norm_rope;
    decltype(&mxgemm_qk_norm_rope_backward_workspace_bytes) qk_norm_rope_backward_workspace_bytes;
    decltype(&mxgemm_qk_norm_rope_backward) qk_norm_rope_backward;
    decltype(&mxgemm_logprobs) logprobs;
    decltype(&mxgemm_logprobs_backward) logprobs_backward;
    decltype(&mxgemm_grad_workspace_bytes) grad_workspace_bytes;
    decltype(&mxgemm_grad_norm) grad_norm;
    decltype(&mxgemm_clip_grads) clip_grads;
};
Entries g_entry;

// Raised as ValueError.
struct BadTensor : std::runtime_error {
    using std::runtime_error::runtime_error;
};

std::string shape_text(std::initializer_list<int64_t> sizes)
{
    std::string s = "(";
    for (const int64_t n : sizes)
        s += std::to_string(n) + ",";
    return s + ")";
}

// An argument: a tensor, or nothing where Python passed None.
const at::Tensor *tensor(PyObject *o, const char *what)
{
    if (o == Py_None)
        return nullptr;
    if (!THPVariable_CheckExact(o) && !THPVariable_Check(o))
        throw BadTensor(std::string(what) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

// What the tensor that sets a call's sizes says about the others.
struct Sizes {
    int64_t rows, cols, stride;
    at::ScalarType dtype;
    c10::Device device = c10::Device(c10::kCPU);
    int in_dtype;
    const void *ptr;

    at::TensorOptions options(at::ScalarType t) const { return at::TensorOptions().dtype(t).device(device); }
};

int in_dtype(at::ScalarType t, const char *what)
{
    if (t == at::kBFloat16)
        return MXGEMM_IN_BF16;
    if (t == at::kFloat)
        return MXGEMM_IN_F32;
    throw BadTensor(std::string(what) + ": unsupported dtype (float32 or bfloat16)");
}

void check_device(const at::Tensor &t, const char *what)
{
    if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
        throw BadTensor(std::string(what) + " must be on the current CUDA device");
}

Sizes matrix(PyObject *o, const char *what)
{
    const at::Tensor *t = tensor(o, what);
    if (!t || t->dim() != 2)
        throw BadTensor(std::string(what) + " must be a 2-D CUDA tensor");
    check_device(*t, what);
    if (t->stride(1) != 1)
        throw BadTensor(std::string(what) + " must have contiguous rows");
    Sizes s;
    s.rows = t->size(0);
    s.cols = t->size(1);
    s.stride = t->stride(0);
    s.dtype = t->scalar_type();
    s.device = t->device();
    s.in_dtype = in_dtype(s.dtype, what);
    s.ptr = t->const_data_ptr();
    return s;
}

// The address of a tensor that is read, or of one that the call writes: data_ptr() first gives
// a tensor that shares its memory copy-on-write a copy of its own.
void *address(const at::Tensor &t, bool written)
{
    return written ? t.data_ptr() : const_cast<void *>(t.const_data_ptr());
}

struct Rows {
    void *ptr = nullptr;
    int64_t stride = 0;
};

// A further matrix of s's type, or nothing.
Rows in_rows(PyObject *o, const Sizes &s, int64_t rows, int64_t cols, const char *what, bool written = false)
{
    Rows r;
    if (const at::Tensor *t = tensor(o, what)) {
        if (t->dim() != 2 || t->size(0) != rows || t->size(1) != cols || t->scalar_type() != s.dtype ||
            t->device() != s.device || t->stride(1) != 1)
            throw BadTensor(std::string(what) + " must be a " + shape_text({rows, cols}) +
                            " tensor of the same dtype and device, with contiguous rows");
        r.ptr = address(*t, written);
        r.stride = t->stride(0);
    }
    return r;
}

// An output: the caller's tensor, checked, or (where `make`) a new one; a strong reference.
struct Out {
    PyObject *object = nullptr;
    void *ptr = nullptr;

    Out() = default;
    Out(const Out &) = delete;
    Out &operator=(const Out &) = delete;
    ~Out() { Py_XDECREF(object); }
    PyObject *release()
    {
        PyObject *o = object;
        object = nullptr;
        return o;
    }
};

void *dense_ptr(const at::Tensor &t, std::initializer_list<int64_t> sizes, at::ScalarType dtype, c10::Device device,
                const char *what)
{
    if (t.sizes() != c10::IntArrayRef(sizes.begin(), sizes.size()) || t.scalar_type() != dtype ||
        t.device() != device || !t.is_contiguous())
        throw BadTensor(std::string(what) + " must be a contiguous " + shape_text(sizes) + " tensor of dtype " +
                        c10::toString(dtype) + " on the inputs' device");
    return t.data_ptr();
}

void output(Out &out, PyObject *o, bool make, std::initializer_list<int64_t> sizes, at::ScalarType dtype,
            const Sizes &s, const char *what)
{
    if (const at::Tensor *t = tensor(o, what)) {
        out.ptr = dense_ptr(*t, sizes, dtype, s.device, what);
        Py_INCREF(o);
        out.object = o;
    } else if (make) {
        at::Tensor n = at::empty(c10::IntArrayRef(sizes.begin(), sizes.size()), s.options(dtype));
        out.ptr = n.data_ptr();
        out.object = THPVariable_Wrap(std::move(n));
        if (!out.object)
            throw python_error();
    } else {
        Py_INCREF(Py_None);
        out.object = Py_None;
    }
}

// Codes and scales of an MX output, made where they are missing.
void mx_output(Out &codes, Out &scales, PyObject *c, PyObject *sc, int fmt, bool tiled, int64_t rows, int64_t K,
               const Sizes &s, const char *what)
{
    if (fmt == 0 && (c != Py_None || sc != Py_None || tiled))
        throw BadTensor(std::string(what) + ": an MX output needs a format");
    const int64_t code_bytes = fmt == MXGEMM_FMT_MXFP8_E4M3 ? K : K / 2;
    output(codes, c, fmt != 0, {rows, code_bytes}, at::kByte, s, "codes");
    if (tiled)
        output(scales, sc, fmt != 0, {static_cast<int64_t>(g_entry.sf_bytes(rows, K))}, at::kByte, s, "scales");
    else
        output(scales, sc, fmt != 0, {rows, K / 32}, at::kByte, s, "scales");
}

// A dense tensor of n elements, whatever its shape.
void *flat(PyObject *o, int64_t n, at::ScalarType dtype, const Sizes &s, const char *what)
{
    const at::Tensor *t = tensor(o, what);
    if (!t)
        return nullptr;
    if (t->numel() != n || t->scalar_type() != dtype || t->device() != s.device || !t->is_contiguous())
        throw BadTensor(std::string(what) + " must be a contiguous tensor of " + std::to_string(n) +
                        " elements of dtype " + c10::toString(dtype) + " on the inputs' device");
    return t->data_ptr();
}

// The norm's weight.
const void *weight_of(PyObject *o, const Sizes &s, int *dtype)
{
    const at::Tensor *t = tensor(o, "weight");
    if (!t || t->dim() != 1 || t->size(0) != s.cols || t->device() != s.device || !t->is_contiguous())
        throw BadTensor("weight must be a contiguous " + shape_text({s.cols}) + " tensor on the inputs' device");
    *dtype = in_dtype(t->scalar_type(), "weight");
    return t->const_data_ptr();
}

// The caller's workspace, or one for this call: torch's allocator reuses its memory in
// the order of the stream that it was allocated on, which is the one that is launched on.
struct Workspace {
    at::Tensor held;
    void *ptr = nullptr;
    size_t bytes = 0;

    Workspace(PyObject *o, size_t need, const Sizes &s)
    {
        if (const at::Tensor *t = tensor(o, "workspace")) {
            if (t->device() != s.device || !t->is_contiguous())
                throw BadTensor("workspace must be a contiguous tensor on the inputs' device");
            ptr = t->data_ptr();
            bytes = t->nbytes();
        } else if (need > 0) {
            held = at::empty({static_cast<int64_t>(need)}, s.options(at::kByte));
            ptr = held.data_ptr();
            bytes = need;
        }
    }
};

void *current_stream(const Sizes &s) { return c10::cuda::getCurrentCUDAStream(s.device.index()).stream(); }

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw python_error();
    return v;
}

// A format or an activation; numbers past an int are as unknown to the library as -1.
int code(PyObject *o)
{
    const int64_t v = integer(o);
    return v == static_cast<int>(v) ? static_cast<int>(v) : -1;
}

bool truth(PyObject *o)
{
    const int t = PyObject_IsTrue(o);
    if (t < 0)
        throw python_error();
    return t != 0;
}

// The outputs of call(), an entry point of the library: it runs without the
// interpreter's lock, since a launch waits while the stream's queue is full.
template <typename F, typename... O>
PyObject *result(F call, O &...out)
{
    struct Unlocked {
        PyThreadState *const state = PyEval_SaveThread();
        ~Unlocked() { PyEval_RestoreThread(state); }
    };
    int status;
    {
        const Unlocked unlocked;
        status = call();
    }
    if (status != MXGEMM_OK)
        return PyLong_FromLong(status);
    PyObject *t = PyTuple_New(sizeof...(O));
    Py_ssize_t i = 0;
    if (t)
        (PyTuple_SET_ITEM(t, i++, out.release()), ...);
    return t;
}

using Args = PyObject *const *;

// (x, weight, eps, residual, fmt, tiled, plain, h, y, codes, scales, rstd)
PyObject *rmsnorm(Args a)
{
    const Sizes s = matrix(a[0], "x");
    int wt = 0;
    const void *w = weight_of(a[1], s, &wt);
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred())
        throw python_error();
    const Rows r = in_rows(a[3], s, s.rows, s.cols, "residual");
    const int fmt = code(a[4]);
    const bool tiled = truth(a[5]), plain = truth(a[6]);
    Out h, y, codes, scales, rstd;
    output(h, a[7], r.ptr != nullptr, {s.rows, s.cols}, s.dtype, s, "h");
    output(y, a[8], plain, {s.rows, s.cols}, s.dtype, s, "y");
    mx_output(codes, scales, a[9], a[10], fmt, tiled, s.rows, s.cols, s, "rmsnorm");
    output(rstd, a[11], true, {s.rows}, at::kFloat, s, "rstd");
    const auto call = [&] {
        return g_entry.rmsnorm(s.in_dtype, s.ptr, s.stride, r.ptr, r.stride, w, wt, static_cast<float>(eps), s.rows,
                               s.cols, h.ptr, y.ptr, fmt, codes.ptr, static_cast<uint8_t *>(scales.ptr),
                               static_cast<float *>(rstd.ptr), tiled ? MXGEMM_QUANT_SF_TILED : 0, current_stream(s));
    };
    return result(call, h, y, codes, scales, rstd);
}

// (dy, h, rstd, weight, dh, dx, dweight, workspace)
PyObject *rmsnorm_backward(Args a)
{
    const Sizes s = matrix(a[0], "dy");
    const Rows h = in_rows(a[1], s, s.rows, s.cols, "h"), dh = in_rows(a[4], s, s.rows, s.cols, "dh");
    int wt = 0;
    const void *w = weight_of(a[3], s, &wt);
    Out rstd, dx, dw;
    output(rstd, a[2], false, {s.rows}, at::kFloat, s, "rstd");
    output(dx, a[5], true, {s.rows, s.cols}, s.dtype, s, "dx");
    output(dw, a[6], true, {s.cols}, at::kFloat, s, "dweight");
    const Workspace ws(a[7], g_entry.rmsnorm_backward_workspace_bytes(s.rows, s.cols), s);
    const auto call = [&] {
        return g_entry.rmsnorm_backward(s.in_dtype, s.ptr, s.stride, h.ptr, h.stride,
                                        static_cast<const float *>(rstd.ptr), w, wt, dh.ptr, dh.stride, s.rows,
                                        s.cols, dx.ptr, static_cast<float *>(dw.ptr), ws.ptr, ws.bytes,
                                        current_stream(s));
    };
    return result(call, dx, dw);
}

// gate and up have one stride
void check_strides(const Sizes &s, int64_t gate, int64_t up)
{
    if (s.rows > 1 && gate != up)
        throw BadTensor("gate and up must have the same row stride");
}

// (gate, up, act, fmt, tiled, plain, keep, y, codes, scales, kept_codes, kept_scales)
PyObject *glu(Args a)
{
    const Sizes s = matrix(a[0], "gate");
    const Rows up = in_rows(a[1], s, s.rows, s.cols, "up");
    if (!up.ptr)
        throw BadTensor("up is missing");
    check_strides(s, s.stride, up.stride);
    const int act = code(a[2]), fmt = code(a[3]);
    const bool tiled = truth(a[4]), plain = truth(a[5]);
    const bool keep = truth(a[6]) || a[10] != Py_None || a[11] != Py_None;
    Out y, codes, scales, kc, ks;
    output(y, a[7], plain, {s.rows, s.cols}, s.dtype, s, "y");
    mx_output(codes, scales, a[8], a[9], fmt, tiled, s.rows, s.cols, s, "glu");
    mx_output(kc, ks, a[10], a[11], keep ? MXGEMM_FMT_MXFP8_E4M3 : 0, false, s.rows, 2 * s.cols, s, "glu");
    const auto call = [&] {
        return g_entry.glu(act, s.in_dtype, s.ptr, up.ptr, s.stride, s.rows, s.cols, y.ptr, fmt, codes.ptr,
                           static_cast<uint8_t *>(scales.ptr), tiled ? MXGEMM_QUANT_SF_TILED : 0, kc.ptr,
                           static_cast<uint8_t *>(ks.ptr), current_stream(s));
    };
    return result(call, y, codes, scales, kc, ks);
}

// (dy, act, gate, up, kept_codes, kept_scales, fmt, tiled, plain, recompute, dgu, codes, scales, a)
PyObject *glu_backward(Args a)
{
    const Sizes s = matrix(a[0], "dy");
    const int act = code(a[1]), fmt = code(a[6]);
    const Rows gate = in_rows(a[2], s, s.rows, s.cols, "gate"), up = in_rows(a[3], s, s.rows, s.cols, "up");
    check_strides(s, gate.stride, up.stride);
    const bool tiled = truth(a[7]), plain = truth(a[8]), recompute = truth(a[9]);
    Out kc, ks, dgu, codes, scales, again;
    output(kc, a[4], false, {s.rows, 2 * s.cols}, at::kByte, s, "kept_codes");
    output(ks, a[5], false, {s.rows, s.cols / 16}, at::kByte, s, "kept_scales");
    output(dgu, a[10], plain, {s.rows, 2 * s.cols}, s.dtype, s, "dgu");
    mx_output(codes, scales, a[11], a[12], fmt, tiled, s.rows, 2 * s.cols, s, "glu_backward");
    output(again, a[13], recompute, {s.rows, s.cols}, s.dtype, s, "a");
    const auto call = [&] {
        return g_entry.glu_backward(act, s.in_dtype, s.ptr, s.stride, gate.ptr, up.ptr, gate.stride, kc.ptr,
                                    static_cast<const uint8_t *>(ks.ptr), s.rows, s.cols, dgu.ptr, fmt, codes.ptr,
                                    static_cast<uint8_t *>(scales.ptr), tiled ? MXGEMM_QUANT_SF_TILED : 0, again.ptr,
                                    current_stream(s));
    };
    return result(call, dgu, codes, scales, again);
}

// (expert_ids, groups, offsets, row_of_slot, slot_of_row, workspace)
PyObject *moe_sort(Args a)
{
    const at::Tensor *ids = tensor(a[0], "expert_ids");
    if (!ids || !ids->is_cuda() || !ids->is_contiguous() ||
        (ids->scalar_type() != at::kInt && ids->scalar_type() != at::kLong))
        throw BadTensor("expert_ids must be a contiguous CUDA int32 or int64 tensor");
    check_device(*ids, "expert_ids");
    const int64_t n = ids->numel(), groups = integer(a[1]);
    Sizes s{};
    s.device = ids->device();
    Out offsets, row, slot;
    // sizes that the library refuses make no tensors
    const bool make = groups >= 1 && groups <= (1 << 20);
    output(offsets, a[2], make, {groups + 1}, at::kLong, s, "offsets");
    output(row, a[3], true, {n}, at::kInt, s, "row_of_slot");
    output(slot, a[4], true, {n}, at::kInt, s, "slot_of_row");
    const Workspace ws(a[5], g_entry.moe_sort_workspace_bytes(n, groups), s);
    const auto call = [&] {
        return g_entry.moe_sort(ids->const_data_ptr(), static_cast<int>(ids->element_size()), n, groups,
                                static_cast<int64_t *>(offsets.ptr), static_cast<int32_t *>(row.ptr),
                                static_cast<int32_t *>(slot.ptr), ws.ptr, ws.bytes, current_stream(s));
    };
    return result(call, offsets, row, slot);
}

// Slots of a token of a row_of_slot table, and the table's address.
int64_t slots_of(PyObject *o, int64_t tokens, const Sizes &s, const int32_t **table)
{
    const at::Tensor *t = tensor(o, "row_of_slot");
    const int64_t n = t ? t->numel() : 0;
    if (tokens < 1 || n < tokens || n % tokens != 0)
        throw BadTensor("row_of_slot must hold the same number of slots for every token");
    *table = static_cast<const int32_t *>(flat(o, n, at::kInt, s, "row_of_slot"));
    return n / tokens;
}

// (x, row_of_slot, fmt, rows, scales)
PyObject *moe_dispatch(Args a)
{
    const Sizes s = matrix(a[0], "x");
    const int32_t *table = nullptr;
    const int64_t topk = slots_of(a[1], s.rows, s, &table), n = topk * s.rows;
    const int fmt = code(a[2]);
    Out rows, scales;
    if (fmt == MXGEMM_FMT_BF16) {
        output(rows, a[3], true, {n, s.cols}, at::kBFloat16, s, "rows");
        if (a[4] != Py_None)
            throw BadTensor("BF16 rows have no scales");
        output(scales, a[4], false, {}, at::kByte, s, "scales");
    } else {
        mx_output(rows, scales, a[3], a[4], fmt, false, n, s.cols, s, "moe_dispatch");
    }
    const auto call = [&] {
        return g_entry.moe_dispatch(s.in_dtype, s.ptr, s.stride, s.rows, topk, s.cols, table, fmt, rows.ptr,
                                    static_cast<uint8_t *>(scales.ptr), current_stream(s));
    };
    return result(call, rows, scales);
}

// (y, row_of_slot, topk, weights, add, out)
PyObject *moe_combine(Args a)
{
    const Sizes s = matrix(a[0], "y");
    const int64_t topk = integer(a[2]);
    if (topk < 1 || s.rows % topk != 0)
        throw BadTensor("y must have one row for each of the tokens * topk slots");
    const int64_t tokens = s.rows / topk;
    const int32_t *table = static_cast<const int32_t *>(flat(a[1], s.rows, at::kInt, s, "row_of_slot"));
    const float *w = static_cast<const float *>(flat(a[3], s.rows, at::kFloat, s, "weights"));
    const Rows add = in_rows(a[4], s, tokens, s.cols, "add");
    Out out;
    output(out, a[5], true, {tokens, s.cols}, s.dtype, s, "out");
    const auto call = [&] {
        return g_entry.moe_combine(s.in_dtype, s.ptr, s.stride, tokens, topk, s.cols, table, w, add.ptr, add.stride,
                                   out.ptr, current_stream(s));
    };
    return result(call, out);
}

// (dout, y, row_of_slot, weights, dy, dweights)
PyObject *moe_combine_backward(Args a)
{
    const Sizes s = matrix(a[0], "dout");
    const int32_t *table = nullptr;
    const int64_t topk = slots_of(a[2], s.rows, s, &table), n = topk * s.rows;
    const Rows y = in_rows(a[1], s, n, s.cols, "y");
    const float *w = static_cast<const float *>(flat(a[3], n, at::kFloat, s, "weights"));
    Out dy, dw;
    output(dy, a[4], true, {n, s.cols}, s.dtype, s, "dy");
    if (a[5] != Py_None || !w) {  // any shape of n elements
        dw.ptr = flat(a[5], n, at::kFloat, s, "dweights");
        Py_INCREF(a[5]);
        dw.object = a[5];
    } else {
        at::Tensor t = at::empty(THPVariable_Unpack(a[3]).sizes(), s.options(at::kFloat));
        dw.ptr = t.data_ptr();
        dw.object = THPVariable_Wrap(std::move(t));
        if (!dw.object)
            throw python_error();
    }
    const auto call = [&] {
        return g_entry.moe_combine_backward(s.in_dtype, s.ptr, s.stride, y.ptr, y.stride, s.rows, topk, s.cols, table,
                                            w, dy.ptr, static_cast<float *>(dw.ptr), current_stream(s));
    };
    return result(call, dy, dw);
}

// ---- the operators of a whole model

float number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return static_cast<float>(v);
}

// A torch dtype, or `otherwise` for None.
at::ScalarType dtype_of(PyObject *o, at::ScalarType otherwise, const char *what)
{
    if (o == Py_None)
        return otherwise;
    if (!THPDtype_Check(o))
        throw BadTensor(std::string(what) + " must be a torch dtype");
    const at::ScalarType t = reinterpret_cast<THPDtype *>(o)->scalar_type;
    in_dtype(t, what);
    return t;
}

// Whole numbers of 32 or 64 bits, `n` of them (n < 0: any number).
struct Ids {
    const void *ptr = nullptr;
    int64_t count = 0;
    int bytes = 0;
    c10::Device device = c10::Device(c10::kCPU);
};

Ids ids_of(PyObject *o, int64_t n, const Sizes *s, const char *what)
{
    Ids r;
    const at::Tensor *t = tensor(o, what);
    if (!t)
        return r;
    if (!t->is_contiguous() || (t->scalar_type() != at::kInt && t->scalar_type() != at::kLong) ||
        (n >= 0 && t->numel() != n) || (s && t->device() != s->device))
        throw BadTensor(std::string(what) + " must be a contiguous int32 or int64 tensor" +
                        (n >= 0 ? " of " + std::to_string(n) + " elements" : "") + " on the inputs' device");
    check_device(*t, what);
    r.ptr = t->const_data_ptr();
    r.count = t->numel();
    r.bytes = static_cast<int>(t->element_size());
    r.device = t->device();
    return r;
}

// (ids, table, scale, dtype, out)
PyObject *embed(Args a)
{
    const Sizes s = matrix(a[1], "table");
    const Ids ids = ids_of(a[0], -1, &s, "ids");
    if (!ids.ptr && ids.count == 0)
        throw BadTensor("ids must hold at least one id");
    const float scale = number(a[2]);
    const at::Tensor *to = tensor(a[4], "out");
    const at::ScalarType dt = to && a[3] == Py_None ? to->scalar_type() : dtype_of(a[3], s.dtype, "dtype");
    const int out_dtype = in_dtype(dt, "out");
    Out out;
    output(out, a[4], true, {ids.count, s.cols}, dt, s, "out");
    const auto call = [&] {
        return g_entry.embed(s.in_dtype, s.ptr, s.stride, s.rows, s.cols, ids.ptr, ids.bytes, ids.count, scale,
                             out_dtype, out.ptr, current_stream(s));
    };
    return result(call, out);
}

// (dy, ids, vocab, scale, dtype, add, dtable, workspace)
PyObject *embed_backward(Args a)
{
    const Sizes s = matrix(a[0], "dy");
    const Ids ids = ids_of(a[1], s.rows, &s, "ids");
    const int64_t vocab = integer(a[2]);
    const float scale = number(a[3]);
    const at::Tensor *given = tensor(a[6], "dtable");
    given = given ? given : tensor(a[5], "add");
    const at::ScalarType dt = given && a[4] == Py_None ? given->scalar_type() : dtype_of(a[4], at::kFloat, "dtype");
    const int out_dtype = in_dtype(dt, "dtable");
    Out add, dtable;
    output(add, a[5], false, {vocab, s.cols}, dt, s, "add");
    // sizes that the library refuses make no tensor
    output(dtable, a[6], vocab >= 1 && vocab < (1ll << 30), {vocab, s.cols}, dt, s, "dtable");
    const Workspace ws(a[7], g_entry.embed_backward_workspace_bytes(s.rows, vocab, s.cols), s);
    const auto call = [&] {
        return g_entry.embed_backward(s.in_dtype, s.ptr, s.stride, ids.ptr, ids.bytes, s.rows, vocab, s.cols, scale,
                                      add.ptr, out_dtype, dtable.ptr, ws.ptr, ws.bytes, current_stream(s));
    };
    return result(call, dtable);
}

// [tokens, heads, D] with contiguous values.
struct HeadsTensor {
    void *ptr = nullptr;
    int64_t token = 0, head = 0;
};

HeadsTensor heads_of(const at::Tensor &t, const char *what, bool written)
{
    if (t.dim() != 3 || t.stride(2) != 1)
        throw BadTensor(std::string(what) + " must be a 3-D CUDA tensor [tokens, heads, D] with contiguous heads");
    check_device(t, what);
    HeadsTensor h;
    h.ptr = address(t, written);
    h.token = t.stride(0);
    h.head = t.stride(1);
    return h;
}

Sizes heads_sizes(PyObject *o, const char *what)
{
    const at::Tensor *t = tensor(o, what);
    if (!t)
        throw BadTensor(std::string(what) + " is missing");
    heads_of(*t, what, false);
    Sizes s{};
    s.rows = t->size(0);
    s.stride = t->size(1);  // heads
    s.cols = t->size(2);
    s.dtype = t->scalar_type();
    s.device = t->device();
    s.in_dtype = in_dtype(s.dtype, what);
    return s;
}

HeadsTensor heads_like(PyObject *o, const Sizes &s, const char *what, bool written = false)
{
    const at::Tensor *t = tensor(o, what);
    if (!t)
        return HeadsTensor();
    if (t->dim() != 3 || t->size(0) != s.rows || t->size(1) != s.stride || t->size(2) != s.cols ||
        t->scalar_type() != s.dtype || t->device() != s.device)
        throw BadTensor(std::string(what) + " must be a " + shape_text({s.rows, s.stride, s.cols}) +
                        " tensor of the same dtype and device");
    return heads_of(*t, what, written);
}

// The caller's strided heads, or new dense ones.
HeadsTensor heads_output(Out &out, PyObject *o, const Sizes &s, const char *what)
{
    if (o != Py_None) {
        const HeadsTensor h = heads_like(o, s, what, true);
        Py_INCREF(o);
        out.object = o;
        return h;
    }
    output(out, o, true, {s.rows, s.stride, s.cols}, s.dtype, s, what);
    HeadsTensor h;
    h.ptr = out.ptr;
    h.token = s.stride * s.cols;
    h.head = s.cols;
    return h;
}

// What both directions take besides the heads: weights, angles, positions.
struct Turn {
    const void *q = nullptr, *k = nullptr;
    int weight_dtype = 0;
    const float *rope = nullptr;
    int64_t rope_rows = 0, rotary = 0;
    Ids positions;
    int64_t q_heads, k_heads;
    uint32_t flags;

    bool norm() const { return q || k; }
    Turn(const Sizes &s, PyObject *count, PyObject *q_weight, PyObject *k_weight, PyObject *table, PyObject *at,
         PyObject *interleaved)
    {
        q_heads = integer(count);
        k_heads = s.stride - q_heads;
        int other = 0;
        if (q_weight != Py_None)
            q = weight_of(q_weight, s, &weight_dtype);
        if (k_weight != Py_None)
            k = weight_of(k_weight, s, &other);
        if (q && k && weight_dtype != other)
            throw BadTensor("q_weight and k_weight must have the same dtype");
        weight_dtype = q ? weight_dtype : other;
        if (const at::Tensor *t = tensor(table, "rope")) {
            if (t->dim() != 2 || t->scalar_type() != at::kFloat || t->device() != s.device || !t->is_contiguous())
                throw BadTensor("rope must be a contiguous 2-D float32 tensor on the inputs' device");
            rope = static_cast<const float *>(t->const_data_ptr());
            rope_rows = t->size(0);
            rotary = t->size(1);
        }
        positions = ids_of(at, s.rows, &s, "positions");
        flags = truth(interleaved) ? MXGEMM_ROPE_INTERLEAVED : 0;
    }
};

// (x, q_heads, q_weight, k_weight, eps, rope, positions, interleaved, y, rstd)
PyObject *qk_norm_rope(Args a)
{
    const Sizes s = heads_sizes(a[0], "x");
    const HeadsTensor x = heads_like(a[0], s, "x");
    const Turn t(s, a[1], a[2], a[3], a[5], a[6], a[7]);
    const float eps = number(a[4]);
    Out y, rstd;
    const HeadsTensor to = heads_output(y, a[8], s, "y");
    output(rstd, a[9], t.norm(), {s.rows, s.stride}, at::kFloat, s, "rstd");
    const auto call = [&] {
        return g_entry.qk_norm_rope(s.in_dtype, x.ptr, x.token, x.head, s.rows, t.q_heads, t.k_heads, s.cols, t.q, t.k,
                                    t.weight_dtype, eps, t.rope, t.rope_rows, t.rotary, t.positions.ptr,
                                    t.positions.bytes, t.flags, to.ptr, to.token, to.head,
                                    static_cast<float *>(rstd.ptr), current_stream(s));
    };
    return result(call, y, rstd);
}

// (dy, x, rstd, q_heads, q_weight, k_weight, rope, positions, interleaved, dx, dq_weight, dk_weight, workspace)
PyObject *qk_norm_rope_backward(Args a)
{
    const Sizes s = heads_sizes(a[0], "dy");
    const HeadsTensor dy = heads_like(a[0], s, "dy"), x = heads_like(a[1], s, "x");
    const Turn t(s, a[3], a[4], a[5], a[6], a[7], a[8]);
    Out rstd, dx, dq, dk;
    output(rstd, a[2], false, {s.rows, s.stride}, at::kFloat, s, "rstd");
    const HeadsTensor to = heads_output(dx, a[9], s, "dx");
    output(dq, a[10], t.q != nullptr, {s.cols}, at::kFloat, s, "dq_weight");
    output(dk, a[11], t.k != nullptr, {s.cols}, at::kFloat, s, "dk_weight");
    const Workspace ws(a[12], t.norm() ? g_entry.qk_norm_rope_backward_workspace_bytes(s.rows, s.stride, s.cols) : 0, s);
    const auto call = [&] {
        return g_entry.qk_norm_rope_backward(
            s.in_dtype, dy.ptr, dy.token, dy.head, x.ptr, x.token, x.head, static_cast<const float *>(rstd.ptr), s.rows,
            t.q_heads, t.k_heads, s.cols, t.q, t.k, t.weight_dtype, t.rope, t.rope_rows, t.rotary, t.positions.ptr,
            t.positions.bytes, t.flags, to.ptr, to.token, to.head, static_cast<float *>(dq.ptr),
            static_cast<float *>(dk.ptr), ws.ptr, ws.bytes, current_stream(s));
    };
    return result(call, dx, dq, dk);
}

// (logits, targets, scale, top, logprob, entropy, stats, top_ids, top_logprobs)
PyObject *logprobs(Args a)
{
    const Sizes s = matrix(a[0], "logits");
    const Ids targets = ids_of(a[1], s.rows, &s, "targets");
    const float scale = number(a[2]);
    const int64_t top = integer(a[3]);
    const bool make = top >= 1 && top <= 1024;  // numbers that the library refuses make no tensors
    Out logprob, entropy, stats, ids, values;
    output(logprob, a[4], targets.ptr != nullptr, {s.rows}, at::kFloat, s, "logprob");
    const bool asked = a[5] == Py_True, none = a[5] == Py_False;
    output(entropy, asked || none ? Py_None : a[5], asked, {s.rows}, at::kFloat, s, "entropy");
    output(stats, a[6], true, {s.rows, 2}, at::kFloat, s, "stats");
    output(ids, a[7], make, {s.rows, top}, at::kLong, s, "top_ids");
    output(values, a[8], make, {s.rows, top}, at::kFloat, s, "top_logprobs");
    const auto call = [&] {
        return g_entry.logprobs(s.in_dtype, s.ptr, s.stride, s.rows, s.cols, scale, targets.ptr, targets.bytes,
                                static_cast<float *>(logprob.ptr), static_cast<float *>(entropy.ptr),
                                static_cast<float *>(stats.ptr), top, static_cast<int64_t *>(ids.ptr),
                                static_cast<float *>(values.ptr), current_stream(s));
    };
    return result(call, logprob, entropy, stats, ids, values);
}

// (logits, targets, stats, dlogprob, entropy, dentropy, scale, dlogits)
PyObject *logprobs_backward(Args a)
{
    const Sizes s = matrix(a[0], "logits");
    const Ids targets = ids_of(a[1], s.rows, &s, "targets");
    const float *g = static_cast<const float *>(flat(a[3], s.rows, at::kFloat, s, "dlogprob"));
    const float *entropy = static_cast<const float *>(flat(a[4], s.rows, at::kFloat, s, "entropy"));
    const float *h = static_cast<const float *>(flat(a[5], s.rows, at::kFloat, s, "dentropy"));
    const float scale = number(a[6]);
    Out stats, dlogits;
    output(stats, a[2], false, {s.rows, 2}, at::kFloat, s, "stats");
    int64_t stride = s.cols;
    if (a[7] != Py_None) {  // the caller's, with its own stride
        const Rows r = in_rows(a[7], s, s.rows, s.cols, "dlogits", true);
        stride = r.stride;
        dlogits.ptr = r.ptr;
        Py_INCREF(a[7]);
        dlogits.object = a[7];
    } else {
        output(dlogits, a[7], true, {s.rows, s.cols}, s.dtype, s, "dlogits");
    }
    const auto call = [&] {
        return g_entry.logprobs_backward(s.in_dtype, s.ptr, s.stride, s.rows, s.cols, scale, targets.ptr,
                                         targets.bytes, static_cast<const float *>(stats.ptr), g, entropy, h,
                                         dlogits.ptr, stride, current_stream(s));
    };
    return result(call, dlogits);
}

// A list or tuple of gradients as host arrays.
struct Grads {
    std::vector<void *> ptr;
    std::vector<int64_t> n;
    std::vector<int> dtype;

    Grads() = default;
    // `like`: another list, of the same shapes and strides.
    Grads(PyObject *list, const char *what, bool written, PyObject *like = nullptr)
    {
        if (!PyList_Check(list) && !PyTuple_Check(list))
            throw BadTensor(std::string(what) + " must be a list or tuple of tensors");
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(list);
        if (like && PySequence_Fast_GET_SIZE(like) != count)
            throw BadTensor(std::string(what) + " must hold a tensor for every gradient");
        ptr.reserve(count);
        n.reserve(count);
        dtype.reserve(count);
        const c10::DeviceIndex device = c10::cuda::current_device();
        for (Py_ssize_t i = 0; i < count; ++i) {
            const at::Tensor *t = tensor(PySequence_Fast_GET_ITEM(list, i), what);
            if (!t)
                throw BadTensor(std::string(what) + ": an entry is None");
            if (!t->is_cuda() || t->get_device() != device)
                throw BadTensor(std::string(what) + " must be on the current CUDA device");
            if (!t->is_non_overlapping_and_dense())
                throw BadTensor(std::string(what) + " must be dense tensors");
            if (like) {
                const at::Tensor &g = THPVariable_Unpack(PySequence_Fast_GET_ITEM(like, i));
                if (t->sizes() != g.sizes() || (t->strides() != g.strides() && !(t->is_contiguous() && g.is_contiguous())))
                    throw BadTensor(std::string(what) + " must have the gradients' shapes and strides");
            }
            ptr.push_back(address(*t, written));
            n.push_back(t->numel());
            dtype.push_back(in_dtype(t->scalar_type(), what));
        }
    }
};

// Sizes of a call on a list: nothing but the device.
Sizes current_sizes()
{
    Sizes s{};
    s.device = c10::Device(c10::kCUDA, c10::cuda::current_device());
    return s;
}

// (grads, norm, workspace)
PyObject *grad_norm(Args a)
{
    const Grads g(a[0], "grads", false);
    const Sizes s = current_sizes();
    const int64_t n = static_cast<int64_t>(g.n.size());
    Out norm;
    output(norm, a[1], true, {1}, at::kFloat, s, "norm");
    const Workspace ws(a[2], g_entry.grad_workspace_bytes(n), s);
    const auto call = [&] {
        return g_entry.grad_norm(n, g.ptr.data(), g.n.data(), g.dtype.data(), static_cast<float *>(norm.ptr), ws.ptr,
                                 ws.bytes, current_stream(s));
    };
    return result(call, norm);
}

// (grads, max_norm, out, norm, workspace)
PyObject *clip_grads(Args a)
{
    const bool apart = a[2] != Py_None;
    const Grads g(a[0], "grads", !apart);
    const float max_norm = number(a[1]);
    const Grads to = apart ? Grads(a[2], "out", true, a[0]) : Grads();
    const Sizes s = current_sizes();
    const int64_t n = static_cast<int64_t>(g.n.size());
    Out norm;
    output(norm, a[3], true, {1}, at::kFloat, s, "norm");
    const Workspace ws(a[4], g_entry.grad_workspace_bytes(n), s);
    const auto call = [&] {
        return g_entry.clip_grads(n, g.ptr.data(), g.n.data(), g.dtype.data(),
                                  apart ? to.ptr.data() : nullptr,
                                  apart ? to.dtype.data() : nullptr, max_norm, static_cast<float *>(norm.ptr), ws.ptr,
                                  ws.bytes, current_stream(s));
    };
    return result(call, norm);
}

// One Python entry: argument count, C++ exceptions to Python ones.
template <PyObject *(*F)(Args), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    if (count != N) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", N, count);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const BadTensor &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// The library's entry points, as addresses in the order of Entries.
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    constexpr Py_ssize_t kEntries = sizeof(Entries) / sizeof(void *);
    void *p[kEntries];
    if (count != kEntries) {
        PyErr_Format(PyExc_TypeError, "%zd addresses expected, %zd given", kEntries, count);
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < kEntries; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (!p[i]) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "an entry point's address is missing");
            return nullptr;
        }
    }
    static_assert(sizeof p == sizeof g_entry, "function and object pointers have one size");
    memcpy(&g_entry, p, sizeof p);
    Py_RETURN_NONE;
}

#define ROWOP(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(bind)), METH_FASTCALL, nullptr},
    ROWOP(rmsnorm, 12),
    ROWOP(rmsnorm_backward, 8),
    ROWOP(glu, 12),
    ROWOP(glu_backward, 14),
    ROWOP(moe_sort, 6),
    ROWOP(moe_dispatch, 5),
    ROWOP(moe_combine, 6),
    ROWOP(moe_combine_backward, 6),
    ROWOP(embed, 5),
    ROWOP(embed_backward, 8),
    ROWOP(qk_norm_rope, 10),
    ROWOP(qk_norm_rope_backward, 13),
    ROWOP(logprobs, 9),
    ROWOP(logprobs_backward, 8),
    ROWOP(grad_norm, 3),
    ROWOP(clip_grads, 5),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_rowops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rowops() { return PyModule_Create(&g_module); }
