// calls.cpp -- the Python calls of the training-step operators (fp8, embedding,
// gradnorm, activation, norm, loss), as an extension module on torch's tensors.
//
// Each function checks its tensors, allocates what the caller did not give,
// and calls the C entry point of libwc.so on the current stream of the tensors'
// GPU.  These calls are made many times per step on small tensors, where the
// host is what takes the time.  Host time on the GB300's Grace, against the
// same steps in Python through ctypes: one-token 8-bit layer (two calls) 24 ->
// 9 us, where its kernels take 6.8; layer forward and backward (six) 75 -> 31;
// embedding lookup 11.3 -> 4.0, gradient 20 -> 7.3; clipping 21 -> 12.
//
// The entry points reach this module as addresses (setup()), so it works with
// whichever build of libwc.so the process has loaded.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/StringUtil.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "wc.h"

namespace {

// ---------------------------------------------------------------------------
// the library
// ---------------------------------------------------------------------------

struct Library {
    decltype(&wc_last_error) last_error;
    decltype(&wc_grad_norm_workspace) grad_norm_workspace;
    decltype(&wc_grad_norm) grad_norm;
    decltype(&wc_grad_clip) grad_clip;
    decltype(&wc_embedding) embedding;
    decltype(&wc_embedding_grad_workspace) embedding_grad_workspace;
    decltype(&wc_embedding_grad) embedding_grad;
    decltype(&wc_fp8_quant) fp8_quant;
    decltype(&wc_fp8_matmul) fp8_matmul;
    decltype(&wc_fp8_dequant) fp8_dequant;
    decltype(&wc_activation) activation;
    decltype(&wc_activation_grad) activation_grad;
    decltype(&wc_rms_norm) rms_norm;
    decltype(&wc_rms_norm_grad_workspace) rms_norm_grad_workspace;
    decltype(&wc_rms_norm_grad) rms_norm_grad;
    decltype(&wc_cross_entropy_workspace) cross_entropy_workspace;
    decltype(&wc_cross_entropy) cross_entropy;
    decltype(&wc_cross_entropy_grad_workspace) cross_entropy_grad_workspace;
    decltype(&wc_cross_entropy_grad) cross_entropy_grad;
};
Library lib;
PyObject *wc_error;  // binding.WcError

[[noreturn]] void raise(PyObject *type, const std::string &message) {
    PyErr_SetString(type, message.c_str());
    throw python_error();
}

template <typename... Parts>
[[noreturn]] void bad_value(const Parts &...parts) {
    raise(PyExc_ValueError, c10::str(parts...));
}

template <typename... Parts>
[[noreturn]] void bad_type(const Parts &...parts) {
    raise(PyExc_TypeError, c10::str(parts...));
}

void check(const char *name, int64_t status) {
    if (status >= 0) return;
    PyObject *e = PyObject_CallFunction(wc_error, "sis", name, int(status), lib.last_error());
    if (e != nullptr) {
        PyErr_SetObject(wc_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

// ---------------------------------------------------------------------------
// arguments
// ---------------------------------------------------------------------------

void arguments(const char *name, Py_ssize_t given, Py_ssize_t wanted) {
    if (given != wanted) bad_type(name, " takes ", wanted, " arguments, got ", given);
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) bad_type(name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

double real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

at::ScalarType dtype(PyObject *o, const char *name) {
    if (!THPDtype_Check(o)) bad_type(name, " must be a torch.dtype, got ", Py_TYPE(o)->tp_name);
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

int float_type(at::ScalarType t, const char *name) {
    if (t == at::kFloat) return WC_F32;
    if (t == at::kBFloat16) return WC_BF16;
    bad_type(name, " must be float32 or bfloat16, got ", t);
}

void on_gpu(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) bad_value(name, " must be a CUDA tensor");
}

void on_device(const at::Tensor &t, const char *name, at::Device device) {
    if (t.device() != device) bad_value(name, " is on ", t.device(), ", expected ", device);
}

// Row stride of a matrix [rows, >= cols] whose rows are consecutive values.
int64_t row_stride(const at::Tensor &t, const char *name, int64_t rows, int64_t cols) {
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) < cols)
        bad_value(name, " has shape ", t.sizes(), ", expected [", rows, ", ", cols, "]");
    if (t.size(1) > 1 && t.stride(1) != 1) bad_value(name, " must have consecutive values in a row");
    if (rows <= 1) return t.size(1);
    if (t.stride(0) < t.size(1)) bad_value(name, " must not have overlapping rows");
    return t.stride(0);
}

// A tensor of activations [.., columns] as a matrix: one of two dimensions whose
// rows are consecutive values, or a contiguous one of any.
struct Rows {
    void *data;
    int64_t rows, cols, ld;
    int type;
};
Rows rows_of(const at::Tensor &t, const char *name) {
    on_gpu(t, name);
    const int type = float_type(t.scalar_type(), name);
    if (t.dim() < 1) bad_value(name, " must have a dimension of columns");
    const int64_t cols = t.size(-1);
    if (t.dim() == 2) return {t.data_ptr(), t.size(0), cols, row_stride(t, name, t.size(0), cols), type};
    if (!t.is_contiguous()) bad_value(name, " must be a matrix or contiguous");
    int64_t rows = 1;
    for (int64_t d = 0; d + 1 < t.dim(); ++d) rows *= t.size(d);
    return {t.data_ptr(), rows, cols, cols, type};
}

// One of the same shape, type and GPU as another.
Rows rows_like(PyObject *o, const char *name, const at::Tensor &like) {
    const at::Tensor &t = tensor(o, name);
    on_device(t, name, like.device());
    if (t.scalar_type() != like.scalar_type()) bad_type(name, " must be ", like.scalar_type(), ", got ", t.scalar_type());
    if (t.sizes() != like.sizes()) bad_value(name, " has shape ", t.sizes(), ", expected ", like.sizes());
    return rows_of(t, name);
}

// A contiguous vector of values of a row.
const at::Tensor &vector_of(PyObject *o, const char *name, int64_t n, at::Device device) {
    const at::Tensor &t = tensor(o, name);
    on_device(t, name, device);
    if (t.numel() != n) bad_value(name, " has shape ", t.sizes(), ", expected ", n, " values");
    if (!t.is_contiguous()) bad_value(name, " must be contiguous");
    return t;
}

const at::Tensor &floats_of(PyObject *o, const char *name, int64_t n, at::Device device) {
    const at::Tensor &t = vector_of(o, name, n, device);
    if (t.scalar_type() != at::kFloat) bad_type(name, " must be float32, got ", t.scalar_type());
    return t;
}

// The calls stand outside autograd.  A tensor that they write to gets a new
// version, so that a backward pass that saved its values finds it changed; an
// input whose gradient ends here is told of.
void written(const at::Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

void ends_gradient(const at::Tensor &t, const char *call, const char *name) {
    if (!t.requires_grad() || !c10::GradMode::is_enabled()) return;
    const std::string m = c10::str(call, " stands outside autograd: no gradient will reach ", name,
                                   " through its result (torch.no_grad() or ", name,
                                   ".detach() says that this is meant)");
    if (PyErr_WarnEx(PyExc_UserWarning, m.c_str(), 1) < 0) throw python_error();
}

void *stream_of(at::Device device) {
    return c10::cuda::getCurrentCUDAStream(device.index()).stream();
}

// A new tensor on a GPU, without the dispatcher's microsecond.
at::Tensor new_tensor(at::IntArrayRef shape, at::ScalarType type, at::Device device) {
    return at::detail::empty_cuda(shape, type, device, std::nullopt);
}

at::Tensor bytes_on(at::Device device, int64_t bytes) {
    if (device.is_cuda()) return new_tensor({bytes}, at::kByte, device);
    return at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(device));
}

const at::Tensor &token_ids(PyObject *o, at::Device device, int *type) {
    const at::Tensor &ids = tensor(o, "ids");
    if (!ids.is_contiguous()) bad_value("ids must be contiguous");
    if (ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong)
        bad_type("ids must be int32 or int64, got ", ids.scalar_type());
    on_device(ids, "ids", device);
    *type = ids.scalar_type() == at::kLong ? WC_I64 : WC_I32;
    return ids;
}

// ---------------------------------------------------------------------------
// embedding
// ---------------------------------------------------------------------------

// (table, ids, scale, first_row, out or None) -> out
PyObject *embedding(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("embedding", n, 5);
    const at::Tensor &table = tensor(args[0], "table");
    if (table.dim() != 2) bad_value("table must be a matrix, got shape ", table.sizes());
    int id_type;
    const at::Tensor &ids = token_ids(args[1], table.device(), &id_type);
    on_gpu(table, "table");
    const int type = float_type(table.scalar_type(), "table");
    const int64_t V = table.size(0), D = table.size(1), tokens = ids.numel();
    const int64_t ld_table = row_stride(table, "table", V, D);
    const c10::cuda::CUDAGuard guard(table.device());
    at::Tensor out;
    int64_t ld_out = D;
    if (args[4] == Py_None) {
        c10::SmallVector<int64_t, 4> shape(ids.sizes().begin(), ids.sizes().end());
        shape.push_back(D);
        out = new_tensor(shape, table.scalar_type(), table.device());
    } else {
        out = tensor(args[4], "out");
        if (out.scalar_type() != table.scalar_type())
            bad_type("out must be ", table.scalar_type(), ", got ", out.scalar_type());
        on_device(out, "out", table.device());
        if (out.dim() == 2 && out.size(1) != D)
            bad_value("out has shape ", out.sizes(), ", expected [", tokens, ", ", D, "]");
        ld_out = row_stride(out, "out", tokens, D);
    }
    ends_gradient(table, "embedding.lookup", "table");
    check("wc_embedding",
          lib.embedding(table.data_ptr(), type, ld_table, ids.data_ptr(), id_type, tokens,
                        integer(args[3]), V, D, float(real(args[2])), out.data_ptr(), ld_out,
                        stream_of(table.device())));
    if (args[4] != Py_None) written(out);
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// (dy, ids, rows, scale, first_row, out or None, out_dtype or None, accumulate) -> out
PyObject *embedding_grad(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("embedding_grad", n, 8);
    const at::Tensor &dy = tensor(args[0], "dy");
    if (dy.dim() < 1) bad_value("dy must have a dimension of columns");
    on_gpu(dy, "dy");
    int id_type;
    const at::Tensor &ids = token_ids(args[1], dy.device(), &id_type);
    const int64_t V = integer(args[2]), D = dy.size(-1), tokens = ids.numel();
    const int dy_type = float_type(dy.scalar_type(), "dy");
    int64_t ld_dy = D;
    if (dy.dim() == 2) {
        ld_dy = row_stride(dy, "dy", tokens, D);
    } else if (dy.sizes().slice(0, dy.dim() - 1) != ids.sizes() || !dy.is_contiguous()) {
        bad_value("dy has shape ", dy.sizes(), ", expected ", ids.sizes(), " and columns, contiguous");
    }
    const c10::cuda::CUDAGuard guard(dy.device());
    const bool accumulate = truth(args[7]);
    at::Tensor out;
    int64_t ld_out = D;
    if (args[5] == Py_None) {
        if (accumulate) bad_value("accumulate needs the gradient to add to as out");
        if (V < 0) bad_value("rows = ", V, " must not be negative");
        const at::ScalarType type = args[6] == Py_None ? dy.scalar_type() : dtype(args[6], "out_dtype");
        float_type(type, "out_dtype");
        out = new_tensor({V, D}, type, dy.device());
    } else {
        out = tensor(args[5], "out");
        if (args[6] != Py_None && out.scalar_type() != dtype(args[6], "out_dtype"))
            bad_type("out must be ", dtype(args[6], "out_dtype"), ", got ", out.scalar_type());
        if (out.dim() == 2 && out.size(1) != D)
            bad_value("out has shape ", out.sizes(), ", expected [", V, ", ", D, "]");
        on_device(out, "out", dy.device());
        ld_out = row_stride(out, "out", V, D);
    }
    const int out_type = float_type(out.scalar_type(), "out");
    ends_gradient(dy, "embedding.grad", "dy");
    const int64_t bytes = lib.embedding_grad_workspace(tokens, V, D);
    check("wc_embedding_grad_workspace", bytes);
    const at::Tensor workspace = bytes_on(dy.device(), bytes > 16 ? bytes : 16);
    check("wc_embedding_grad",
          lib.embedding_grad(dy.data_ptr(), dy_type, ld_dy, ids.data_ptr(), id_type, tokens,
                             integer(args[4]), V, D, float(real(args[3])), accumulate ? 1 : 0,
                             out.data_ptr(), out_type, ld_out, workspace.data_ptr(),
                             workspace.numel(), stream_of(dy.device())));
    if (args[5] != Py_None) written(out);
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------
// gradient norm
// ---------------------------------------------------------------------------

// The wc_span list of a tuple of dense tensors on one GPU (*device, if the tuple
// is the first of its call).  Made at each call, so it is where the tensors are now.
using Spans = c10::SmallVector<wc_span, 32>;
Spans spans_of(PyObject *tuple, const char *name, std::optional<at::Device> *device) {
    if (!PyTuple_Check(tuple)) bad_type(name, " must be a tuple of tensors, got ", Py_TYPE(tuple)->tp_name);
    const Py_ssize_t count = PyTuple_GET_SIZE(tuple);
    if (count > 0x7FFFFFFF) bad_value("a list of ", count, " tensors is too long");
    Spans spans;
    spans.reserve(size_t(count));
    for (Py_ssize_t i = 0; i < count; ++i) {
        const at::Tensor &t = tensor(PyTuple_GET_ITEM(tuple, i), name);
        if (!t.is_cuda()) bad_value(name, "[", i, "] must be a CUDA tensor");
        if (!device->has_value()) *device = t.device();
        else if (t.device() != **device) bad_value(name, "[", i, "] is on ", t.device(), ", expected ", **device);
        if (!t.is_contiguous()) bad_value(name, "[", i, "] must be contiguous");
        const bool f32 = t.scalar_type() == at::kFloat;
        if (!f32 && t.scalar_type() != at::kBFloat16)
            bad_type(name, "[", i, "] must be float32 or bfloat16, got ", t.scalar_type());
        spans.push_back({t.numel() > 0 ? t.data_ptr() : nullptr, t.numel(), f32 ? WC_F32 : WC_BF16, 0});
    }
    return spans;
}

// (tuple of tensors) -> their GPU, or None if there are none
PyObject *grad_list(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("grad_list", n, 1);
    std::optional<at::Device> device;
    spans_of(args[0], "tensors", &device);
    if (!device.has_value()) Py_RETURN_NONE;
    return THPDevice_New(*device);
    END_HANDLE_TH_ERRORS
}

// (tensors, where their values go or None (in place), clip, max_norm, eps,
//  stats or None) -> stats
PyObject *grad_norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("grad_norm", n, 6);
    std::optional<at::Device> found;
    const Spans spans = spans_of(args[0], "tensors", &found);
    if (!found.has_value()) bad_value("an empty list has no GPU to run on");
    const bool in_place = args[1] == Py_None;
    const Spans dst = in_place ? Spans() : spans_of(args[1], "out", &found);
    if (!in_place && dst.size() != spans.size())
        bad_value("out has ", dst.size(), " tensors, expected ", spans.size());
    const int count = int(spans.size());
    const bool clip = truth(args[2]);
    const at::Device device = *found;
    const c10::cuda::CUDAGuard guard(device);
    at::Tensor stats;
    const int64_t values = clip ? 2 : 1;
    if (args[5] == Py_None) {
        stats = new_tensor({values}, at::kFloat, device);
    } else {
        stats = tensor(args[5], "stats");
        on_gpu(stats, "stats");
        on_device(stats, "stats", device);
        if (stats.scalar_type() != at::kFloat) bad_type("stats must be float32, got ", stats.scalar_type());
        if (!stats.is_contiguous()) bad_value("stats must be contiguous");
        if (stats.numel() != values)
            bad_value("stats has ", stats.numel(), " elements, expected ", values);
    }
    const at::Tensor workspace = bytes_on(device, lib.grad_norm_workspace(count));
    auto *out = static_cast<float *>(stats.data_ptr());
    if (clip)
        check("wc_grad_clip", lib.grad_clip(spans.data(), in_place ? nullptr : dst.data(), count,
                                            real(args[3]), real(args[4]), out, workspace.data_ptr(),
                                            workspace.numel(), stream_of(device)));
    else
        check("wc_grad_norm", lib.grad_norm(spans.data(), count, out, workspace.data_ptr(),
                                            workspace.numel(), stream_of(device)));
    if (args[5] != Py_None) written(stats);
    if (clip) {
        PyObject *to = in_place ? args[0] : args[1];
        for (int i = 0; i < count; ++i) written(THPVariable_Unpack(PyTuple_GET_ITEM(to, i)));
    }
    return THPVariable_Wrap(stats);
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------
// 8-bit matrices
// ---------------------------------------------------------------------------

constexpr int64_t kBlock = 128;

int64_t ceil_to(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }

int64_t checked_block_rows(int64_t b) {
    if (b != 1 && b != kBlock) bad_value("block_rows must be 1 or 128, got ", b);
    return b;
}

// A matrix [rows, cols] in 8 bits, as a call needs it.  Python holds it as its
// parts (codes, scales, rows, cols, block_rows), or, for codes and scales in one
// buffer of bytes, (buffer, None, rows, cols, block_rows): the tensors themselves,
// so that a copy of the parts is a copy of the matrix.  Addresses are taken, and
// sizes checked, at each call.
struct Matrix8 {
    uint8_t *q = nullptr;
    float *s = nullptr;
    int64_t ld_codes = 0, ld_scales = 0, rows = 0, cols = 0, block_rows = 0;
    at::Device device = at::Device(at::kCPU);

    // Codes, then scales, in one buffer.  The scales of a block start on 16
    // bytes, where a product fetches them four at a time.  Returns the place of
    // the scales and, in *bytes, the buffer's size.
    int64_t lay_out(int64_t *bytes) {
        ld_codes = ceil_to(cols, 16);
        ld_scales = ceil_to((rows + block_rows - 1) / block_rows, 4);
        const int64_t scales_at = ceil_to(rows * ld_codes, 16);
        *bytes = scales_at + blocks(cols) * ld_scales * 4;
        return scales_at;
    }
    void in_buffer(const at::Tensor &buffer) {
        int64_t bytes;
        const int64_t scales_at = lay_out(&bytes);
        if (buffer.scalar_type() != at::kByte || !buffer.is_contiguous() || buffer.numel() != bytes)
            bad_value("the buffer of an 8-bit matrix [", rows, ", ", cols, "] must be ", bytes,
                      " contiguous bytes, got ", buffer.scalar_type(), " ", buffer.sizes());
        device = buffer.device();
        q = static_cast<uint8_t *>(buffer.data_ptr());
        s = reinterpret_cast<float *>(q + scales_at);
    }
    void in_tensors(const at::Tensor &codes, const at::Tensor &scales) {
        if (codes.scalar_type() != at::kFloat8_e4m3fn)
            bad_type("codes must be float8_e4m3fn, got ", codes.scalar_type());
        if (scales.scalar_type() != at::kFloat)
            bad_type("scales must be float32, got ", scales.scalar_type());
        if (scales.device() != codes.device())
            bad_value("scales are on ", scales.device(), ", codes on ", codes.device());
        ld_codes = row_stride(codes, "codes", rows, cols);
        ld_scales = row_stride(scales, "scales", blocks(cols), (rows + block_rows - 1) / block_rows);
        // there is no second row to be apart from
        if (rows <= 1 || codes.size(1) == 0) ld_codes = ceil_to(cols, 16);
        device = codes.device();
        q = static_cast<uint8_t *>(codes.data_ptr());
        s = static_cast<float *>(scales.data_ptr());
    }
    static Matrix8 of(PyObject *t) {
        if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != 5) bad_type("not an 8-bit matrix");
        Matrix8 m;
        m.rows = integer(PyTuple_GET_ITEM(t, 2));
        m.cols = integer(PyTuple_GET_ITEM(t, 3));
        m.block_rows = checked_block_rows(integer(PyTuple_GET_ITEM(t, 4)));
        const at::Tensor &codes = tensor(PyTuple_GET_ITEM(t, 0), "codes");
        if (PyTuple_GET_ITEM(t, 1) == Py_None) m.in_buffer(codes);
        else m.in_tensors(codes, tensor(PyTuple_GET_ITEM(t, 1), "scales"));
        return m;
    }
};

// A new matrix's buffer.
at::Tensor make(Matrix8 *m, int64_t rows, int64_t cols, int64_t block_rows, at::Device device) {
    if (rows < 0 || cols < 0) bad_value("rows = ", rows, ", cols = ", cols, " must not be negative");
    m->rows = rows;
    m->cols = cols;
    m->block_rows = block_rows;
    int64_t bytes;
    m->lay_out(&bytes);
    const at::Tensor buffer = bytes_on(device, bytes);
    m->in_buffer(buffer);
    return buffer;
}

// Its parts.
PyObject *described(const Matrix8 &m, const at::Tensor &buffer) {
    PyObject *t = Py_BuildValue("NOLLL", THPVariable_Wrap(buffer), Py_None, (long long)m.rows,
                                (long long)m.cols, (long long)m.block_rows);
    if (t == nullptr) throw python_error();
    return t;
}

// (rows, cols, block_rows, device) -> parts
PyObject *fp8_empty(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("fp8_empty", n, 4);
    if (!THPDevice_Check(args[3])) bad_type("device must be a torch.device");
    Matrix8 m;
    const at::Tensor buffer = make(&m, integer(args[0]), integer(args[1]),
                                   checked_block_rows(integer(args[2])),
                                   reinterpret_cast<THPDevice *>(args[3])->device);
    return described(m, buffer);
    END_HANDLE_TH_ERRORS
}

// (codes, scales, rows, cols, block_rows) -> parts
PyObject *fp8_view(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("fp8_view", n, 5);
    Matrix8 m;
    m.block_rows = checked_block_rows(integer(args[4]));
    const at::Tensor &codes = tensor(args[0], "codes"), &scales = tensor(args[1], "scales");
    m.rows = integer(args[2]);
    m.cols = integer(args[3]);
    m.in_tensors(codes, scales);
    PyObject *t = Py_BuildValue("OOOOO", args[0], args[1], args[2], args[3], args[4]);
    if (t == nullptr) throw python_error();
    return t;
    END_HANDLE_TH_ERRORS
}

void quantize(const at::Tensor &x, const Matrix8 &q, const Matrix8 &qt, bool square) {
    const int64_t rows = x.size(0), cols = x.size(1);
    const int64_t ld = row_stride(x, "x", rows, cols);
    check("wc_fp8_quant",
          lib.fp8_quant(x.data_ptr(), float_type(x.scalar_type(), "x"), rows, cols, ld, square ? 1 : 0,
                        q.q, q.ld_codes, q.s, q.ld_scales, qt.q, qt.ld_codes, qt.s,
                        qt.ld_scales, stream_of(x.device())));
}

const at::Tensor &matrix(PyObject *o) {
    const at::Tensor &x = tensor(o, "x");
    if (x.dim() != 2) bad_value("x must be a matrix, got shape ", x.sizes());
    return x;
}

// (x, rows, columns, block_rows) -> (parts or None, parts or None)
PyObject *fp8_quantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("fp8_quantize", n, 4);
    const at::Tensor &x = matrix(args[0]);
    const bool rows = truth(args[1]), columns = truth(args[2]);
    const int64_t block_rows = checked_block_rows(integer(args[3]));
    if (!rows && !columns) bad_value("neither rows nor columns asked for");
    on_gpu(x, "x");
    float_type(x.scalar_type(), "x");
    // (a weight's codes are kept beside it, and its gradient comes from backward)
    if (block_rows == 1) ends_gradient(x, "fp8.quantize", "x");
    const c10::cuda::CUDAGuard guard(x.device());
    Matrix8 q, qt;
    at::Tensor buffer, buffer_t;
    if (rows) buffer = make(&q, x.size(0), x.size(1), block_rows, x.device());
    if (columns) buffer_t = make(&qt, x.size(1), x.size(0), block_rows, x.device());
    quantize(x, q, qt, block_rows == kBlock);
    PyObject *a = rows ? described(q, buffer) : Py_NewRef(Py_None);
    PyObject *b = columns ? described(qt, buffer_t) : Py_NewRef(Py_None);
    return Py_BuildValue("NN", a, b);
    END_HANDLE_TH_ERRORS
}

// (x, parts or None, parts of the transposed matrix or None) -> None
PyObject *fp8_quantize_into(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("fp8_quantize_into", n, 3);
    const at::Tensor &x = matrix(args[0]);
    on_gpu(x, "x");
    Matrix8 q, qt;
    if (args[1] != Py_None) q = Matrix8::of(args[1]);
    if (args[2] != Py_None) qt = Matrix8::of(args[2]);
    const Matrix8 &any = args[1] != Py_None ? q : qt;
    on_device(x, "x", any.device);
    if (args[1] != Py_None && (q.rows != x.size(0) || q.cols != x.size(1)))
        bad_value("x has shape ", x.sizes(), ", the 8-bit matrix [", q.rows, ", ", q.cols, "]");
    if (args[2] != Py_None && (qt.rows != x.size(1) || qt.cols != x.size(0)))
        bad_value("x has shape ", x.sizes(), ", the transposed 8-bit matrix [", qt.rows, ", ", qt.cols, "]");
    const c10::cuda::CUDAGuard guard(x.device());
    quantize(x, q, qt, any.block_rows == kBlock);
    for (PyObject *parts : {args[1], args[2]})
        for (int i = 0; parts != Py_None && i < 2; ++i)
            if (PyTuple_GET_ITEM(parts, i) != Py_None) written(THPVariable_Unpack(PyTuple_GET_ITEM(parts, i)));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// (parts of a, parts of b, out or None, out_dtype, accumulate) -> out
PyObject *fp8_matmul(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("fp8_matmul", n, 5);
    const Matrix8 a = Matrix8::of(args[0]), b = Matrix8::of(args[1]);
    if (a.cols != b.cols) bad_value("a has ", a.cols, " columns, b ", b.cols);
    const at::Device device = a.device;
    if (b.device != device) bad_value("b is on ", b.device, ", expected ", device);
    if (!device.is_cuda()) bad_value("the operands must be CUDA tensors");
    const bool accumulate = truth(args[4]);
    const c10::cuda::CUDAGuard guard(device);
    at::Tensor out;
    int64_t ld_out = b.rows;
    if (args[2] == Py_None) {
        if (accumulate) bad_value("accumulate needs the matrix to add to as out");
        const at::ScalarType type = dtype(args[3], "out_dtype");
        float_type(type, "out_dtype");
        out = new_tensor({a.rows, b.rows}, type, device);
    } else {
        out = tensor(args[2], "out");
        if (out.dim() == 2 && out.size(1) != b.rows)
            bad_value("out has shape ", out.sizes(), ", expected [", a.rows, ", ", b.rows, "]");
        on_device(out, "out", device);
        ld_out = row_stride(out, "out", a.rows, b.rows);
    }
    check("wc_fp8_matmul",
          lib.fp8_matmul(a.q, a.ld_codes, a.s, a.ld_scales, int(a.block_rows), b.q, b.ld_codes,
                         b.s, b.ld_scales, int(b.block_rows), a.rows, b.rows, a.cols,
                         out.data_ptr(), float_type(out.scalar_type(), "out"), ld_out,
                         accumulate ? 1 : 0, stream_of(device)));
    if (args[2] != Py_None) written(out);
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// (parts, out or None, out_dtype) -> out
PyObject *fp8_dequantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("fp8_dequantize", n, 3);
    const Matrix8 q = Matrix8::of(args[0]);
    if (!q.device.is_cuda()) bad_value("the 8-bit matrix must be on a GPU");
    const c10::cuda::CUDAGuard guard(q.device);
    at::Tensor out;
    int64_t ld_out = q.cols;
    if (args[1] == Py_None) {
        const at::ScalarType type = dtype(args[2], "out_dtype");
        float_type(type, "out_dtype");
        out = new_tensor({q.rows, q.cols}, type, q.device);
    } else {
        out = tensor(args[1], "out");
        if (out.dim() == 2 && out.size(1) != q.cols)
            bad_value("out has shape ", out.sizes(), ", expected [", q.rows, ", ", q.cols, "]");
        on_device(out, "out", q.device);
        ld_out = row_stride(out, "out", q.rows, q.cols);
    }
    check("wc_fp8_dequant",
          lib.fp8_dequant(q.q, q.ld_codes, q.s, q.ld_scales, int(q.block_rows), q.rows, q.cols, out.data_ptr(),
                          float_type(out.scalar_type(), "out"), ld_out, stream_of(q.device)));
    if (args[1] != Py_None) written(out);
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------
// activations and norms kept in 8 bits
// ---------------------------------------------------------------------------

wc_kept kept_of(const Matrix8 &m) { return {m.q, m.ld_codes, m.s, m.ld_scales}; }

// A matrix [rows, cols] that a forward pass kept.
Matrix8 kept_matrix(PyObject *parts, const char *name, int64_t rows, int64_t cols, at::Device device) {
    const Matrix8 m = Matrix8::of(parts);
    if (m.rows != rows || m.cols != cols || m.block_rows != 1)
        bad_value(name, " is [", m.rows, ", ", m.cols, "] with ", m.block_rows, " rows per scale, expected [", rows,
                  ", ", cols, "] with 1");
    if (m.device != device) bad_value(name, " is on ", m.device, ", expected ", device);
    return m;
}

// (gate, up or None, kind, save, out or None) -> (h, parts of gate or None, parts of up or None)
PyObject *activation(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("activation", n, 5);
    const at::Tensor &gate = tensor(args[0], "gate");
    const Rows g = rows_of(gate, "gate");
    const bool gated = args[1] != Py_None, save = truth(args[3]);
    const Rows u = gated ? rows_like(args[1], "up", gate) : Rows{nullptr, 0, 0, g.cols, 0};
    const int kind = int(integer(args[2]));
    const at::Device device = gate.device();
    const c10::cuda::CUDAGuard guard(device);
    at::Tensor h;
    Rows o;
    if (args[4] == Py_None) {
        h = new_tensor(gate.sizes(), gate.scalar_type(), device);
        o = {h.data_ptr(), g.rows, g.cols, g.cols, g.type};
    } else {
        o = rows_like(args[4], "out", gate);
        h = tensor(args[4], "out");
    }
    ends_gradient(gate, "activation.forward", "gate");
    if (gated) ends_gradient(tensor(args[1], "up"), "activation.forward", "up");
    Matrix8 kg, ku;
    at::Tensor buffer, buffer_up;
    if (save) buffer = make(&kg, g.rows, g.cols, 1, device);
    if (save && gated) buffer_up = make(&ku, g.rows, g.cols, 1, device);
    const wc_kept k = kept_of(kg), k_up = kept_of(ku);
    check("wc_activation",
          lib.activation(g.data, g.ld, u.data, u.ld, g.type, kind, g.rows, g.cols, o.data, o.ld, save ? &k : nullptr,
                         save && gated ? &k_up : nullptr, stream_of(device)));
    if (args[4] != Py_None) written(h);
    PyObject *a = save ? described(kg, buffer) : Py_NewRef(Py_None);
    PyObject *b = save && gated ? described(ku, buffer_up) : Py_NewRef(Py_None);
    return Py_BuildValue("NNN", THPVariable_Wrap(h), a, b);
    END_HANDLE_TH_ERRORS
}

// (dh, kind, parts of gate, parts of up or None) -> (dgate, dup or None)
PyObject *activation_grad(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("activation_grad", n, 4);
    const at::Tensor &dh = tensor(args[0], "dh");
    const Rows d = rows_of(dh, "dh");
    const int kind = int(integer(args[1]));
    const bool gated = args[3] != Py_None;
    const at::Device device = dh.device();
    const Matrix8 kg = kept_matrix(args[2], "the kept gate", d.rows, d.cols, device);
    const Matrix8 ku = gated ? kept_matrix(args[3], "the kept up", d.rows, d.cols, device) : Matrix8();
    const c10::cuda::CUDAGuard guard(device);
    ends_gradient(dh, "activation.backward", "dh");
    const at::Tensor dgate = new_tensor(dh.sizes(), dh.scalar_type(), device);
    at::Tensor dup;
    if (gated) dup = new_tensor(dh.sizes(), dh.scalar_type(), device);
    const wc_kept k = kept_of(kg), k_up = kept_of(ku);
    check("wc_activation_grad",
          lib.activation_grad(d.data, d.ld, d.type, kind, d.rows, d.cols, &k, gated ? &k_up : nullptr,
                              dgate.data_ptr(), d.cols, gated ? dup.data_ptr() : nullptr, d.cols, stream_of(device)));
    return Py_BuildValue("NN", THPVariable_Wrap(dgate), gated ? THPVariable_Wrap(dup) : Py_NewRef(Py_None));
    END_HANDLE_TH_ERRORS
}

// (x, weight, eps, add or None, save) -> (y, total or None, rstd or None, parts or None)
PyObject *rms_norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("rms_norm", n, 5);
    const at::Tensor &x = tensor(args[0], "x");
    const Rows r = rows_of(x, "x");
    const at::Device device = x.device();
    const at::Tensor &weight = vector_of(args[1], "weight", r.cols, device);
    const int weight_type = float_type(weight.scalar_type(), "weight");
    const bool adds = args[3] != Py_None, save = truth(args[4]);
    const Rows a = adds ? rows_like(args[3], "add", x) : Rows{nullptr, 0, 0, r.cols, 0};
    const c10::cuda::CUDAGuard guard(device);
    ends_gradient(x, "norm.rms", "x");
    ends_gradient(weight, "norm.rms", "weight");
    if (adds) ends_gradient(tensor(args[3], "add"), "norm.rms", "add");
    const at::Tensor y = new_tensor(x.sizes(), x.scalar_type(), device);
    at::Tensor total, rstd, buffer;
    if (adds) total = new_tensor(x.sizes(), x.scalar_type(), device);
    Matrix8 m;
    if (save) {
        rstd = new_tensor({r.rows}, at::kFloat, device);
        buffer = make(&m, r.rows, r.cols, 1, device);
    }
    const wc_kept k = kept_of(m);
    check("wc_rms_norm",
          lib.rms_norm(r.data, r.ld, a.data, a.ld, r.type, r.rows, r.cols, weight.data_ptr(), weight_type,
                       real(args[2]), y.data_ptr(), r.cols, adds ? total.data_ptr() : nullptr, r.cols,
                       save ? static_cast<float *>(rstd.data_ptr()) : nullptr, save ? &k : nullptr,
                       stream_of(device)));
    PyObject *t = adds ? THPVariable_Wrap(total) : Py_NewRef(Py_None);
    PyObject *s = save ? THPVariable_Wrap(rstd) : Py_NewRef(Py_None);
    PyObject *q = save ? described(m, buffer) : Py_NewRef(Py_None);
    return Py_BuildValue("NNNN", THPVariable_Wrap(y), t, s, q);
    END_HANDLE_TH_ERRORS
}

// (dy, weight, rstd, parts, add or None, dweight or None, accumulate) -> (dx, dweight)
PyObject *rms_norm_grad(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("rms_norm_grad", n, 7);
    const at::Tensor &dy = tensor(args[0], "dy");
    const Rows d = rows_of(dy, "dy");
    const at::Device device = dy.device();
    const at::Tensor &weight = vector_of(args[1], "weight", d.cols, device);
    const int weight_type = float_type(weight.scalar_type(), "weight");
    const at::Tensor &rstd = floats_of(args[2], "rstd", d.rows, device);
    const Matrix8 m = kept_matrix(args[3], "the kept input", d.rows, d.cols, device);
    const bool adds = args[4] != Py_None, accumulate = truth(args[6]);
    const Rows a = adds ? rows_like(args[4], "add", dy) : Rows{nullptr, 0, 0, d.cols, 0};
    const c10::cuda::CUDAGuard guard(device);
    at::Tensor dweight;
    if (args[5] == Py_None) {
        if (accumulate) bad_value("accumulate needs the gradient to add to as dweight");
        dweight = new_tensor({d.cols}, at::kFloat, device);
    } else {
        dweight = vector_of(args[5], "dweight", d.cols, device);
    }
    ends_gradient(dy, "norm.rms_grad", "dy");
    const at::Tensor dx = new_tensor(dy.sizes(), dy.scalar_type(), device);
    const int64_t bytes = lib.rms_norm_grad_workspace(d.rows, d.cols);
    check("wc_rms_norm_grad_workspace", bytes);
    const at::Tensor workspace = bytes_on(device, bytes > 16 ? bytes : 16);
    const wc_kept k = kept_of(m);
    check("wc_rms_norm_grad",
          lib.rms_norm_grad(d.data, d.ld, a.data, a.ld, d.type, d.rows, d.cols, weight.data_ptr(), weight_type,
                            static_cast<float *>(rstd.data_ptr()), &k, dx.data_ptr(), d.cols, dweight.data_ptr(),
                            float_type(dweight.scalar_type(), "dweight"), accumulate ? 1 : 0, workspace.data_ptr(),
                            workspace.numel(), stream_of(device)));
    if (args[5] != Py_None) written(dweight);
    return Py_BuildValue("NN", THPVariable_Wrap(dx), THPVariable_Wrap(dweight));
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------
// cross entropy
// ---------------------------------------------------------------------------

// x [.., D], weight [V, D] and targets (one per row of x) of both directions.
struct Tokens {
    const at::Tensor &x, &w, &targets;
    int64_t T, V, D, ld_x, ld_w;
    int id_type;
    const uint16_t *px() const { return static_cast<const uint16_t *>(x.data_ptr()); }
    const uint16_t *pw() const { return static_cast<const uint16_t *>(w.data_ptr()); }
};
Tokens tokens_of(PyObject *const *args) {
    const at::Tensor &x = tensor(args[0], "x"), &w = tensor(args[1], "weight"), &y = tensor(args[2], "targets");
    const Rows r = rows_of(x, "x");
    if (r.type != WC_BF16) bad_type("x must be bfloat16, got ", x.scalar_type());
    if (w.scalar_type() != at::kBFloat16) bad_type("weight must be bfloat16, got ", w.scalar_type());
    on_device(w, "weight", x.device());
    if (w.dim() != 2 || w.size(1) != r.cols)
        bad_value("weight has shape ", w.sizes(), ", expected [rows, ", r.cols, "]");
    if (y.scalar_type() != at::kInt && y.scalar_type() != at::kLong)
        bad_type("targets must be int32 or int64, got ", y.scalar_type());
    on_device(y, "targets", x.device());
    if (!y.is_contiguous()) bad_value("targets must be contiguous");
    if (y.numel() != r.rows) bad_value("targets has shape ", y.sizes(), ", expected one for each of ", r.rows, " rows of x");
    return {x, w, y, r.rows, w.size(0), r.cols, r.ld, row_stride(w, "weight", w.size(0), r.cols),
            y.scalar_type() == at::kLong ? WC_I64 : WC_I32};
}

// (x, weight, targets) -> (losses, lse)
PyObject *cross_entropy(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("cross_entropy", n, 3);
    const Tokens t = tokens_of(args);
    const at::Device device = t.x.device();
    const c10::cuda::CUDAGuard guard(device);
    ends_gradient(t.x, "loss.cross_entropy", "x");
    ends_gradient(t.w, "loss.cross_entropy", "weight");
    const at::Tensor losses = new_tensor(t.targets.sizes(), at::kFloat, device);
    const at::Tensor lse = new_tensor(t.targets.sizes(), at::kFloat, device);
    const int64_t bytes = lib.cross_entropy_workspace(t.px(), t.ld_x, t.pw(), t.ld_w, t.T, t.V, t.D);
    check("wc_cross_entropy_workspace", bytes);
    const at::Tensor workspace = bytes_on(device, bytes > 16 ? bytes : 16);
    check("wc_cross_entropy",
          lib.cross_entropy(t.px(), t.ld_x, t.pw(), t.ld_w, t.targets.data_ptr(), t.id_type, t.T, t.V, t.D,
                            static_cast<float *>(losses.data_ptr()), static_cast<float *>(lse.data_ptr()),
                            workspace.data_ptr(), workspace.numel(), stream_of(device)));
    return Py_BuildValue("NN", THPVariable_Wrap(losses), THPVariable_Wrap(lse));
    END_HANDLE_TH_ERRORS
}

// (x, weight, targets, lse, dlosses (tensor or number), dx wanted, dw wanted, dw or None,
//  dw_dtype or None, accumulate) -> (dx or None, dw or None)
PyObject *cross_entropy_grad(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("cross_entropy_grad", n, 10);
    const Tokens t = tokens_of(args);
    const at::Device device = t.x.device();
    const at::Tensor &lse = floats_of(args[3], "lse", t.T, device);
    const float *dlosses = nullptr;
    double dloss = 0.0;
    if (THPVariable_Check(args[4])) {
        const at::Tensor &d = floats_of(args[4], "dlosses", t.T, device);
        ends_gradient(d, "loss.cross_entropy_grad", "dlosses");
        dlosses = static_cast<const float *>(d.data_ptr());
    } else {
        dloss = real(args[4]);
    }
    const bool want_dx = truth(args[5]), want_dw = truth(args[6]), accumulate = truth(args[9]);
    if (!want_dx && !want_dw) bad_value("neither dx nor dw asked for");
    const c10::cuda::CUDAGuard guard(device);
    at::Tensor dx, dw;
    int64_t ld_dw = t.D;
    if (want_dx) dx = new_tensor(t.x.sizes(), at::kBFloat16, device);
    if (!want_dw) {
        if (accumulate || args[7] != Py_None) bad_value("dw is given and not asked for");
    } else if (args[7] == Py_None) {
        if (accumulate) bad_value("accumulate needs the gradient to add to as dw");
        const at::ScalarType type = args[8] == Py_None ? at::kBFloat16 : dtype(args[8], "dw_dtype");
        float_type(type, "dw_dtype");
        dw = new_tensor({t.V, t.D}, type, device);
    } else {
        dw = tensor(args[7], "dw");
        if (args[8] != Py_None && dw.scalar_type() != dtype(args[8], "dw_dtype"))
            bad_type("dw must be ", dtype(args[8], "dw_dtype"), ", got ", dw.scalar_type());
        if (dw.dim() == 2 && dw.size(1) != t.D)
            bad_value("dw has shape ", dw.sizes(), ", expected [", t.V, ", ", t.D, "]");
        on_device(dw, "dw", device);
        ld_dw = row_stride(dw, "dw", t.V, t.D);
    }
    const int dw_type = want_dw ? float_type(dw.scalar_type(), "dw") : WC_BF16;
    const int64_t bytes = lib.cross_entropy_grad_workspace(t.px(), t.ld_x, t.pw(), t.ld_w, t.T, t.V, t.D);
    check("wc_cross_entropy_grad_workspace", bytes);
    const at::Tensor workspace = bytes_on(device, bytes > 16 ? bytes : 16);
    check("wc_cross_entropy_grad",
          lib.cross_entropy_grad(t.px(), t.ld_x, t.pw(), t.ld_w, t.targets.data_ptr(), t.id_type, t.T, t.V, t.D,
                                 static_cast<const float *>(lse.data_ptr()), dlosses, dloss,
                                 want_dx ? dx.data_ptr() : nullptr, WC_BF16, t.D,
                                 want_dw ? dw.data_ptr() : nullptr, dw_type, ld_dw, accumulate ? 1 : 0,
                                 workspace.data_ptr(), workspace.numel(), stream_of(device)));
    if (args[7] != Py_None) written(dw);
    return Py_BuildValue("NN", want_dx ? THPVariable_Wrap(dx) : Py_NewRef(Py_None),
                         want_dw ? THPVariable_Wrap(dw) : Py_NewRef(Py_None));
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------
// module
// ---------------------------------------------------------------------------

// (dict of entry point addresses by name, WcError)
PyObject *setup(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments("setup", n, 2);
    auto entry = [&](const char *name, auto *slot) {
        PyObject *o = PyDict_Check(args[0]) ? PyDict_GetItemString(args[0], name) : nullptr;
        if (o == nullptr) bad_value("no address of ", name);
        *slot = reinterpret_cast<std::remove_reference_t<decltype(*slot)>>(integer(o));
    };
    entry("wc_last_error", &lib.last_error);
    entry("wc_grad_norm_workspace", &lib.grad_norm_workspace);
    entry("wc_grad_norm", &lib.grad_norm);
    entry("wc_grad_clip", &lib.grad_clip);
    entry("wc_embedding", &lib.embedding);
    entry("wc_embedding_grad_workspace", &lib.embedding_grad_workspace);
    entry("wc_embedding_grad", &lib.embedding_grad);
    entry("wc_fp8_quant", &lib.fp8_quant);
    entry("wc_fp8_matmul", &lib.fp8_matmul);
    entry("wc_fp8_dequant", &lib.fp8_dequant);
    entry("wc_activation", &lib.activation);
    entry("wc_activation_grad", &lib.activation_grad);
    entry("wc_rms_norm", &lib.rms_norm);
    entry("wc_rms_norm_grad_workspace", &lib.rms_norm_grad_workspace);
    entry("wc_rms_norm_grad", &lib.rms_norm_grad);
    entry("wc_cross_entropy_workspace", &lib.cross_entropy_workspace);
    entry("wc_cross_entropy", &lib.cross_entropy);
    entry("wc_cross_entropy_grad_workspace", &lib.cross_entropy_grad_workspace);
    entry("wc_cross_entropy_grad", &lib.cross_entropy_grad);
    Py_INCREF(args[1]);
    Py_XSETREF(wc_error, args[1]);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define WC_METHOD(name) \
    { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {WC_METHOD(setup),        WC_METHOD(embedding),    WC_METHOD(embedding_grad),
                         WC_METHOD(grad_list),    WC_METHOD(grad_norm),    WC_METHOD(fp8_empty),    WC_METHOD(fp8_view),
                         WC_METHOD(fp8_quantize), WC_METHOD(fp8_quantize_into), WC_METHOD(fp8_matmul),
                         WC_METHOD(fp8_dequantize), WC_METHOD(activation), WC_METHOD(activation_grad),
                         WC_METHOD(rms_norm),     WC_METHOD(rms_norm_grad), WC_METHOD(cross_entropy),
                         WC_METHOD(cross_entropy_grad),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "wc_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_wc_calls() { return PyModule_Create(&module); }
