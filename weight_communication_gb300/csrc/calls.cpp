// calls.cpp -- the Python calls of the training-step operators (fp8, embedding,
// gradnorm), as an extension module on torch's tensors.
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
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "wc_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_wc_calls() { return PyModule_Create(&module); }
