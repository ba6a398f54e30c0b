// The short way from Python to the microscaled, group-scaled, routing and experts' calls
// (include/mq.h).
//
// A call on a few tokens takes the GPU 3 to 10 us, and its way through Python's own
// checks, ctypes and torch's allocation functions took longer than that. Each function
// here takes the operands as the public function has them, goes through the same checks,
// allocates the outputs and calls the library; it returns None where anything is not as
// it should be (a wrong type or size, another device than the current one, a status that
// is not 0), and the public function, in mx.py or experts.py, then goes its own long way
// to the precise error or the other device. Nothing is launched twice: a None comes
// before the launch, or with an error status of it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/saved_variable.h>

#include <string.h>

#include <mutex>
#include <utility>

#include "../../include/mq.h"

#define MQ_TEXT_(x) #x
#define MQ_TEXT(x) MQ_TEXT_(x)
#define MQ_PYTHON_VERSION MQ_TEXT(PY_MAJOR_VERSION) "." MQ_TEXT(PY_MINOR_VERSION) "."

namespace {

using at::ScalarType;

PyTypeObject* mx_type = nullptr;
PyTypeObject* plan_type = nullptr;
PyTypeObject* w4_type = nullptr;

struct No {};                                      // not this way

void need(bool ok) {
    if (!ok) throw No{};
}

int type_code(ScalarType t) {
    if (t == ScalarType::Float) return MQ_F32;
    if (t == ScalarType::BFloat16) return MQ_BF16;
    need(t == ScalarType::Half);
    return MQ_F16;
}

ScalarType dtype_of(PyObject* o) {
    need(THPDtype_Check(o));
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

const at::Tensor& tensor(PyObject* o) {
    need(THPVariable_Check(o));
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
    need(PyLong_Check(o));
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw No{};
    }
    return v;
}

// The current device and its current stream (torch calls the type of a HIP device CUDA).
struct Here {
    c10::Device device{c10::DeviceType::CUDA, c10::hip::current_device()};
    void* stream() const { return c10::hip::getCurrentHIPStream(device.index()).stream(); }
    bool has(const at::Tensor& t) const { return t.is_cuda() && t.get_device() == device.index(); }
    at::Tensor make(at::IntArrayRef size, ScalarType type) const {
        return at::Tensor(at::detail::empty_cuda(size, type, device, std::nullopt));
    }
};

const at::Tensor& contiguous(const Here& here, const at::Tensor& t, ScalarType type, at::IntArrayRef size) {
    need(t.scalar_type() == type && t.sizes() == size && here.has(t) && t.is_contiguous());
    return t;
}

const at::Tensor& contiguous(const Here& here, PyObject* o, ScalarType type, at::IntArrayRef size) {
    return contiguous(here, tensor(o), type, size);
}

// a strided matrix whose last axis is contiguous
const at::Tensor& input(const Here& here, const at::Tensor& t, int64_t dims) {
    need(t.dim() == dims && here.has(t) && (t.stride(-1) == 1 || t.size(-1) <= 1));
    return t;
}

const at::Tensor& input(const Here& here, PyObject* o, int64_t dims) {
    return input(here, tensor(o), dims);
}

// One of the public named tuples, with all of its items (a tuple type's instance can be made
// with fewer, by tuple.__new__): only then are they read without a check each.
bool whole(PyObject* o, const PyTypeObject* type, Py_ssize_t items) {
    return Py_TYPE(o) == type && PyTuple_GET_SIZE(o) == items;
}

struct Matrix {
    const uint8_t *codes, *scales;
    int64_t rows, cols;
};

Matrix matrix(const Here& here, PyObject* o, int64_t batch = -1) {
    need(whole(o, mx_type, 4));
    Matrix m;
    m.rows = integer(PyTuple_GET_ITEM(o, 2));
    m.cols = integer(PyTuple_GET_ITEM(o, 3));
    const int64_t tiles = (m.rows + 15) / 16, groups = (m.cols + 127) / 128, quads = (groups + 3) / 4;
    const int64_t codes[4] = {batch, tiles, groups, 1024}, scales[4] = {batch, tiles, quads, 256};
    const int skip = batch < 0 ? 1 : 0;
    m.codes = contiguous(here, PyTuple_GET_ITEM(o, 0), ScalarType::Byte, {codes + skip, codes + 4}).const_data_ptr<uint8_t>();
    m.scales = contiguous(here, PyTuple_GET_ITEM(o, 1), ScalarType::Byte, {scales + skip, scales + 4}).const_data_ptr<uint8_t>();
    return m;
}

// the caller's output, or a new one
at::Tensor output(const Here& here, PyObject* o, PyObject* type, at::IntArrayRef size) {
    if (o == Py_None) {
        const ScalarType t = dtype_of(type);
        type_code(t);
        return here.make(size, t);
    }
    const at::Tensor& y = tensor(o);
    type_code(y.scalar_type());
    need(y.sizes() == size && here.has(y) && y.is_contiguous() && reinterpret_cast<uintptr_t>(y.data_ptr()) % 16 == 0);
    return y;
}

// The caller's output, written, which counts as a change of it (a gradient may have kept what it
// held), or the new one.
PyObject* wrapped(PyObject* given, const at::Tensor& y) {
    if (given == Py_None) return THPVariable_Wrap(y);
    if (!y.is_inference()) y.unsafeGetTensorImpl()->bump_version();
    Py_INCREF(given);
    return given;
}

// A named tuple of these (stolen) values.
PyObject* named(PyTypeObject* type, std::initializer_list<PyObject*> values) {
    PyObject* t = type->tp_alloc(type, static_cast<Py_ssize_t>(values.size()));
    Py_ssize_t i = 0;
    for (PyObject* v : values) {
        if (t) PyTuple_SET_ITEM(t, i++, v);
        else Py_XDECREF(v);
    }
    return t;
}

void* data(const at::Tensor& t) { return t.data_ptr(); }

// quantize(x, out)
PyObject* quantize(PyObject* const* a) {
    const Here here;
    const at::Tensor& x = tensor(a[0]);
    const bool batched = x.dim() == 3;
    input(here, a[0], batched ? 3 : 2);
    const int code = type_code(x.scalar_type());
    const int64_t B = batched ? x.size(0) : 1, R = x.size(-2), K = x.size(-1);
    need(K > 0);
    const int64_t tiles = (R + 15) / 16, groups = (K + 127) / 128, quads = (groups + 3) / 4;
    const int64_t cs[4] = {B, tiles, groups, 1024}, ss[4] = {B, tiles, quads, 256};
    const int skip = batched ? 0 : 1;
    at::Tensor codes, scales;
    uint8_t *cp, *sp;
    if (a[1] == Py_None) {
        codes = here.make({cs + skip, cs + 4}, ScalarType::Byte);
        scales = here.make({ss + skip, ss + 4}, ScalarType::Byte);
        cp = static_cast<uint8_t*>(data(codes));
        sp = static_cast<uint8_t*>(data(scales));
    } else {
        const Matrix m = matrix(here, a[1], batched ? B : -1);
        need(m.rows == R && m.cols == K);
        cp = const_cast<uint8_t*>(m.codes);
        sp = const_cast<uint8_t*>(m.scales);
    }
    need(mq_mx_quantize(data(x), code, B, batched ? x.stride(0) : 0, R, x.stride(-2), K, cp, sp, here.stream()) == MQ_OK);
    if (a[1] != Py_None) {
        Py_INCREF(a[1]);
        return a[1];
    }
    return named(mx_type, {THPVariable_Wrap(codes), THPVariable_Wrap(scales), PyLong_FromLongLong(R), PyLong_FromLongLong(K)});
}

// dequantize(a, dtype, out)
PyObject* dequantize(PyObject* const* a) {
    const Here here;
    need(whole(a[0], mx_type, 4));
    const at::Tensor& c = tensor(PyTuple_GET_ITEM(a[0], 0));
    const bool batched = c.dim() == 4;
    const int64_t B = batched ? c.size(0) : 1;
    const Matrix m = matrix(here, a[0], batched ? B : -1);
    const int64_t size[3] = {B, m.rows, m.cols};
    const at::Tensor y = output(here, a[2], a[1], {size + (batched ? 0 : 1), size + 3});
    need(mq_mx_dequantize(m.codes, m.scales, B, m.rows, m.cols, data(y), type_code(y.scalar_type()), here.stream()) == MQ_OK);
    return wrapped(a[2], y);
}

// linear(x, w, bias, out_dtype, y)
PyObject* linear(PyObject* const* a) {
    const Here here;
    const Matrix w = matrix(here, a[1]);
    const float* bias = a[2] == Py_None ? nullptr : contiguous(here, a[2], ScalarType::Float, {w.rows}).const_data_ptr<float>();
    int rc;
    if (Py_TYPE(a[0]) == mx_type) {
        const Matrix x = matrix(here, a[0]);
        need(x.cols == w.cols);
        const at::Tensor y = output(here, a[4], a[3], {x.rows, w.rows});
        rc = mq_mx_gemm(x.codes, x.scales, w.codes, w.scales, x.rows, w.rows, w.cols, bias, data(y), type_code(y.scalar_type()),
                        here.stream());
        need(rc == MQ_OK);
        return wrapped(a[4], y);
    }
    const at::Tensor& x = input(here, a[0], 2);
    need(x.size(1) == w.cols);
    const int64_t M = x.size(0);
    const at::Tensor y = output(here, a[4], a[3], {M, w.rows});
    const size_t bytes = mq_mx_linear_workspace_bytes(M, w.rows, w.cols);
    at::Tensor work;
    if (bytes) work = here.make({static_cast<int64_t>(bytes)}, ScalarType::Byte);
    rc = mq_mx_linear(data(x), type_code(x.scalar_type()), x.stride(0), w.codes, w.scales, M, w.rows, w.cols, bias, data(y),
                      type_code(y.scalar_type()), bytes ? data(work) : nullptr, bytes, here.stream());
    need(rc == MQ_OK);
    return wrapped(a[4], y);
}

// route(logits, k, score, bias, groups, top_groups, group_score, renormalize, scale, ids, weights)
PyObject* route(PyObject* const* a) {
    const Here here;
    const at::Tensor& x = input(here, a[0], 2);
    const int64_t T = x.size(0), E = x.size(1), k = integer(a[1]), groups = integer(a[4]), top = integer(a[5]);
    need(groups > 0 && E % groups == 0 && top > 0 && top <= groups && k > 0 && k <= top * (E / groups));
    const float* bias = a[3] == Py_None ? nullptr : contiguous(here, a[3], ScalarType::Float, {E}).const_data_ptr<float>();
    const int renormalize = PyObject_IsTrue(a[7]);
    need(renormalize >= 0 && PyFloat_Check(a[8]));
    const at::Tensor ids = a[9] == Py_None ? here.make({T, k}, ScalarType::Int) : contiguous(here, a[9], ScalarType::Int, {T, k});
    const at::Tensor weights = a[10] == Py_None ? here.make({T, k}, ScalarType::Float)
                                                : contiguous(here, a[10], ScalarType::Float, {T, k});
    need(mq_route(data(x), type_code(x.scalar_type()), T, x.stride(0), E, bias, static_cast<int>(integer(a[2])), groups, top,
                  static_cast<int>(integer(a[6])), k, renormalize, static_cast<float>(PyFloat_AS_DOUBLE(a[8])),
                  static_cast<int32_t*>(data(ids)), static_cast<float*>(data(weights)), here.stream()) == MQ_OK);
    PyObject* both = PyTuple_New(2);
    if (!both) return nullptr;
    PyTuple_SET_ITEM(both, 0, wrapped(a[9], ids));
    PyTuple_SET_ITEM(both, 1, wrapped(a[10], weights));
    return both;
}

// expert_plan(ids, experts)
PyObject* expert_plan(PyObject* const* a) {
    const Here here;
    const at::Tensor& ids = tensor(a[0]);
    need(ids.dim() == 2 && ids.scalar_type() == ScalarType::Int && here.has(ids) && ids.is_contiguous());
    const int64_t T = ids.size(0), k = ids.size(1), E = integer(a[1]), rows = mq_plan_rows(T, k, E);
    need(rows >= 0);
    const at::Tensor offsets = here.make({E + 1}, ScalarType::Int), row_token = here.make({rows}, ScalarType::Int),
                     row_of = here.make({T, k}, ScalarType::Int);
    need(mq_expert_plan(static_cast<const int32_t*>(data(ids)), T, k, E, static_cast<int32_t*>(data(offsets)),
                        static_cast<int32_t*>(data(row_token)), static_cast<int32_t*>(data(row_of)), here.stream()) == MQ_OK);
    return named(plan_type, {THPVariable_Wrap(offsets), THPVariable_Wrap(row_token), THPVariable_Wrap(row_of)});
}

struct Plan {
    const int32_t *offsets, *row_token, *row_of;
    int64_t T, k, E, rows;
};

Plan plan(const Here& here, const at::Tensor& offsets, const at::Tensor& row_token, const at::Tensor& row_of) {
    need(row_of.dim() == 2 && offsets.dim() == 1);
    Plan p;
    p.T = row_of.size(0);
    p.k = row_of.size(1);
    p.E = offsets.size(0) - 1;
    p.rows = mq_plan_rows(p.T, p.k, p.E);
    need(p.rows >= 0);
    p.offsets = contiguous(here, offsets, ScalarType::Int, {p.E + 1}).const_data_ptr<int32_t>();
    p.row_token = contiguous(here, row_token, ScalarType::Int, {p.rows}).const_data_ptr<int32_t>();
    p.row_of = contiguous(here, row_of, ScalarType::Int, {p.T, p.k}).const_data_ptr<int32_t>();
    return p;
}

Plan plan(const Here& here, PyObject* o) {
    need(whole(o, plan_type, 3));
    return plan(here, tensor(PyTuple_GET_ITEM(o, 0)), tensor(PyTuple_GET_ITEM(o, 1)), tensor(PyTuple_GET_ITEM(o, 2)));
}

// experts_up(x, w_gate, w_up, plan, out_dtype, h)
PyObject* experts_up(PyObject* const* a) {
    const Here here;
    const at::Tensor& x = input(here, a[0], 2);
    const Plan p = plan(here, a[3]);
    const Matrix g = matrix(here, a[1], p.E), u = matrix(here, a[2], p.E);
    need(g.rows == u.rows && g.cols == u.cols && x.size(0) == p.T && x.size(1) == g.cols);
    const at::Tensor h = output(here, a[5], a[4], {p.rows, g.rows});
    const size_t bytes = mq_mx_experts_up_workspace_bytes(p.T, p.k, p.E, g.cols, g.rows);
    at::Tensor work;
    if (bytes) work = here.make({static_cast<int64_t>(bytes)}, ScalarType::Byte);
    need(mq_mx_experts_up(data(x), type_code(x.scalar_type()), x.stride(0), p.T, p.k, p.E, g.cols, g.rows, p.offsets, p.row_token,
                          p.row_of, g.codes, g.scales, u.codes, u.scales, data(h), type_code(h.scalar_type()),
                          bytes ? data(work) : nullptr, bytes, here.stream()) == MQ_OK);
    return wrapped(a[5], h);
}

// experts_down(h, w_down, plan, weights, out_dtype, y)
PyObject* experts_down(PyObject* const* a) {
    const Here here;
    const Plan p = plan(here, a[2]);
    const Matrix w = matrix(here, a[1], p.E);
    const at::Tensor& h = tensor(a[0]);
    contiguous(here, a[0], h.scalar_type(), {p.rows, w.cols});
    const float* weights = contiguous(here, a[3], ScalarType::Float, {p.T, p.k}).const_data_ptr<float>();
    const at::Tensor y = output(here, a[5], a[4], {p.T, w.rows});
    const size_t bytes = mq_mx_experts_down_workspace_bytes(p.T, p.k, p.E, w.rows, w.cols);
    at::Tensor work;
    if (bytes) work = here.make({static_cast<int64_t>(bytes)}, ScalarType::Byte);
    need(mq_mx_experts_down(data(h), type_code(h.scalar_type()), p.T, p.k, p.E, w.rows, w.cols, p.offsets, p.row_of, weights,
                            w.codes, w.scales, data(y), type_code(y.scalar_type()), bytes ? data(work) : nullptr, bytes,
                            here.stream()) == MQ_OK);
    return wrapped(a[5], y);
}

// no gradient is wanted of it, and it carries no tangent of forward mode
const at::Tensor& plain(const at::Tensor& t) {
    need((!t.requires_grad() || !at::GradMode::is_enabled()) && !t._fw_grad(0).defined());
    return t;
}

int group_of(PyObject* o) {
    const int64_t g = PyBool_Check(o) ? 0 : integer(o);
    need(g == 32 || g == 64 || g == 128);
    return static_cast<int>(g);
}

ScalarType scale_type(ScalarType t) {
    need(t == ScalarType::Half || t == ScalarType::BFloat16);
    return t;
}

struct Group4 {
    const uint8_t* codes;
    const void *scales, *zeros;
    ScalarType type;
    int64_t rows, cols;
    int group;
};

struct Sizes4 {
    int64_t c[4], s[5];
    int skip;
    Sizes4(int64_t batch, int64_t rows, int64_t cols, int group)
        : c{batch, (rows + 15) / 16, (cols + 127) / 128, 1024}, s{batch, (rows + 15) / 16, (cols + 511) / 512, 16, 512 / group},
          skip(batch < 0 ? 1 : 0) {}
    at::IntArrayRef codes() const { return {c + skip, c + 4}; }
    at::IntArrayRef scales() const { return {s + skip, s + 5}; }
};

Group4 group4(const Here& here, PyObject* o, int64_t batch = -1) {
    need(whole(o, w4_type, 6));
    Group4 m;
    m.rows = integer(PyTuple_GET_ITEM(o, 3));
    m.cols = integer(PyTuple_GET_ITEM(o, 4));
    m.group = group_of(PyTuple_GET_ITEM(o, 5));
    const Sizes4 size(batch, m.rows, m.cols, m.group);
    m.codes = contiguous(here, PyTuple_GET_ITEM(o, 0), ScalarType::Byte, size.codes()).const_data_ptr<uint8_t>();
    m.type = scale_type(tensor(PyTuple_GET_ITEM(o, 1)).scalar_type());
    m.scales = contiguous(here, PyTuple_GET_ITEM(o, 1), m.type, size.scales()).const_data_ptr();
    PyObject* const z = PyTuple_GET_ITEM(o, 2);
    m.zeros = z == Py_None ? nullptr : contiguous(here, z, m.type, size.scales()).const_data_ptr();
    return m;
}

// a new W4's tensors, and the tuple of them
struct New4 {
    at::Tensor codes, scales, zeros;
    New4(const Here& here, const Sizes4& size, ScalarType type, bool z)
        : codes(here.make(size.codes(), ScalarType::Byte)), scales(here.make(size.scales(), type)) {
        if (z) zeros = here.make(size.scales(), type);
    }
    void* zeros_data() const { return zeros.defined() ? data(zeros) : nullptr; }
    PyObject* tuple(int64_t rows, int64_t cols, int group) const {
        PyObject* z = Py_None;
        if (zeros.defined()) z = THPVariable_Wrap(zeros);
        else Py_INCREF(z);
        return named(w4_type, {THPVariable_Wrap(codes), THPVariable_Wrap(scales), z, PyLong_FromLongLong(rows),
                               PyLong_FromLongLong(cols), PyLong_FromLong(group)});
    }
};

// w4_quantize(x, group, zeros, scale_dtype, out)
PyObject* w4_quantize(PyObject* const* a) {
    const Here here;
    const bool batched = tensor(a[0]).dim() == 3;
    const at::Tensor& x = input(here, a[0], batched ? 3 : 2);
    const int group = group_of(a[1]), z = PyObject_IsTrue(a[2]);
    need(z >= 0 && a[4] == Py_None && x.size(-1) > 0);
    const ScalarType type = scale_type(dtype_of(a[3]));
    const int64_t B = batched ? x.size(0) : 1, R = x.size(-2), K = x.size(-1);
    const New4 w(here, Sizes4(batched ? B : -1, R, K, group), type, z != 0);
    need(mq_w4_quantize(data(x), type_code(x.scalar_type()), B, batched ? x.stride(0) : 0, R, x.stride(-2), K, group,
                        type_code(type), static_cast<uint8_t*>(data(w.codes)), data(w.scales), w.zeros_data(), here.stream()) == MQ_OK);
    return w.tuple(R, K, group);
}

// w4_pack(codes, scales, zeros, group)
PyObject* w4_pack(PyObject* const* a) {
    const Here here;
    const bool batched = tensor(a[0]).dim() == 3;
    const at::Tensor& c = input(here, a[0], batched ? 3 : 2);
    const int group = group_of(a[3]);
    const int64_t B = batched ? c.size(0) : 1, R = c.size(-2), K = c.size(-1), n = (K + group - 1) / group;
    need(c.scalar_type() == ScalarType::Byte && K > 0);
    const ScalarType type = scale_type(tensor(a[1]).scalar_type());
    const int64_t given[3] = {B, R, n};
    const at::IntArrayRef per(given + (batched ? 0 : 1), given + 3);
    const void* const s = contiguous(here, a[1], type, per).const_data_ptr();
    const void* const z = a[2] == Py_None ? nullptr : contiguous(here, a[2], type, per).const_data_ptr();
    const New4 w(here, Sizes4(batched ? B : -1, R, K, group), type, a[2] != Py_None);
    need(mq_w4_pack(c.const_data_ptr<uint8_t>(), B, batched ? c.stride(0) : 0, R, c.stride(-2), K, group, s, z,
                    static_cast<uint8_t*>(data(w.codes)), data(w.scales), w.zeros_data(), here.stream()) == MQ_OK);
    return w.tuple(R, K, group);
}

// w4_dequantize(a, dtype, out)
PyObject* w4_dequantize(PyObject* const* a) {
    const Here here;
    need(whole(a[0], w4_type, 6));
    const at::Tensor& c = tensor(PyTuple_GET_ITEM(a[0], 0));
    const bool batched = c.dim() == 4;
    const int64_t B = batched ? c.size(0) : 1;
    const Group4 m = group4(here, a[0], batched ? B : -1);
    const int64_t size[3] = {B, m.rows, m.cols};
    const at::Tensor y = output(here, a[2], a[1], {size + (batched ? 0 : 1), size + 3});
    need(mq_w4_dequantize(m.codes, m.scales, m.zeros, type_code(m.type), B, m.rows, m.cols, m.group, data(y),
                          type_code(y.scalar_type()), here.stream()) == MQ_OK);
    return wrapped(a[2], y);
}

// The memory from t's first to its last element.
std::pair<uintptr_t, uintptr_t> span(const at::Tensor& t) {
    const uintptr_t first = reinterpret_cast<uintptr_t>(t.const_data_ptr());
    int64_t last = 0;
    for (int64_t i = 0; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
    return {first, t.numel() ? first + (last + 1) * t.element_size() : first};
}

// The caller's output is not memory that is still read.
const at::Tensor& apart(const at::Tensor& y, const at::Tensor& x) {
    const auto a = span(y), b = span(x);
    need(a.second <= b.first || b.second <= a.first);
    return y;
}

// w4_linear(x, w, bias, out_dtype, y)
PyObject* w4_linear(PyObject* const* a) {
    const Here here;
    const at::Tensor& x = plain(input(here, a[0], 2));
    const Group4 w = group4(here, a[1]);
    const float* bias = a[2] == Py_None ? nullptr : plain(contiguous(here, a[2], ScalarType::Float, {w.rows})).const_data_ptr<float>();
    need(x.size(1) == w.cols);
    const int64_t M = x.size(0);
    const int code = type_code(x.scalar_type());
    const at::Tensor y = apart(output(here, a[4], a[3], {M, w.rows}), x);
    const size_t bytes = mq_w4_linear_workspace_bytes(M, w.rows, w.cols, code, w.group);
    at::Tensor work;
    if (bytes) work = here.make({static_cast<int64_t>(bytes)}, ScalarType::Byte);
    need(mq_w4_linear(data(x), code, x.stride(0), w.codes, w.scales, w.zeros, type_code(w.type), w.group, M, w.rows, w.cols, bias,
                      data(y), type_code(y.scalar_type()), bytes ? data(work) : nullptr, bytes, here.stream()) == MQ_OK);
    return wrapped(a[4], y);
}

// w4_experts(x, w, plan, by_token, out_dtype, y)
PyObject* w4_experts(PyObject* const* a) {
    const Here here;
    const at::Tensor& x = plain(input(here, a[0], 2));
    const Plan p = plan(here, a[2]);
    const Group4 w = group4(here, a[1], p.E);
    const int by_token = PyObject_IsTrue(a[3]), code = type_code(x.scalar_type());
    need(by_token >= 0 && x.size(0) == (by_token ? p.T : p.rows) && x.size(1) == w.cols);
    const at::Tensor y = apart(output(here, a[5], a[4], {p.rows, w.rows}), x);
    const size_t bytes = mq_w4_experts_workspace_bytes(p.T, p.k, p.E, w.rows, w.cols, by_token, code, w.group);
    at::Tensor work;
    if (bytes) work = here.make({static_cast<int64_t>(bytes)}, ScalarType::Byte);
    need(mq_w4_experts(data(x), code, x.stride(0), by_token, p.T, p.k, p.E, w.rows, w.cols, p.offsets, p.row_token, w.codes,
                       w.scales, w.zeros, type_code(w.type), w.group, data(y), type_code(y.scalar_type()),
                       bytes ? data(work) : nullptr, bytes, here.stream()) == MQ_OK);
    return wrapped(a[5], y);
}

const float* weights_of(const Here& here, PyObject* o, const Plan& p) {
    return o == Py_None ? nullptr : plain(contiguous(here, o, ScalarType::Float, {p.T, p.k})).const_data_ptr<float>();
}

// (y, dots), or y alone
PyObject* with_dots(PyObject* given, const at::Tensor& y, const at::Tensor& dots) {
    if (!dots.defined()) return wrapped(given, y);
    PyObject* both = PyTuple_New(2);
    if (!both) return nullptr;
    PyTuple_SET_ITEM(both, 0, wrapped(given, y));
    PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(dots));
    return both;
}

// an output of `type`, or of the type `same` where that is None
at::Tensor output_as(const Here& here, PyObject* o, PyObject* type, ScalarType same, at::IntArrayRef size) {
    return o == Py_None && type == Py_None ? here.make(size, same) : output(here, o, type, size);
}

// The two ways, on checked operands; `other` and `dots` may be undefined.
void run_gather(const Here& here, const Plan& p, const at::Tensor& x, const float* weights, const at::Tensor& rows,
                const at::Tensor& other, const at::Tensor& dots) {
    need(mq_experts_gather(data(x), type_code(x.scalar_type()), x.stride(0), p.T, p.k, p.E, x.size(1), p.row_token, p.row_of, weights,
                           data(rows), type_code(rows.scalar_type()), other.defined() ? data(other) : nullptr,
                           other.defined() ? static_cast<float*>(data(dots)) : nullptr, here.stream()) == MQ_OK);
}

void run_combine(const Here& here, const Plan& p, const at::Tensor& rows, const float* weights, const at::Tensor& y,
                 const at::Tensor& other, const at::Tensor& dots) {
    need(mq_experts_combine(data(rows), type_code(rows.scalar_type()), p.T, p.k, p.E, rows.size(1), p.row_of, weights, data(y),
                            type_code(y.scalar_type()), other.defined() ? data(other) : nullptr, other.defined() ? other.stride(0) : 0,
                            other.defined() ? static_cast<float*>(data(dots)) : nullptr, here.stream()) == MQ_OK);
}

const at::Tensor& tokens(const Here& here, const at::Tensor& x, const Plan& p) {
    input(here, x, 2);
    need(x.size(0) == p.T && x.size(1) > 0);
    type_code(x.scalar_type());
    return x;
}

const at::Tensor& plan_rows(const Here& here, const at::Tensor& rows, const Plan& p) {
    input(here, rows, 2);
    need(rows.size(0) == p.rows && rows.size(1) > 0 && rows.is_contiguous());
    type_code(rows.scalar_type());
    return rows;
}

// gather(x, plan, weights, dtype, rows, other)
PyObject* gather(PyObject* const* a) {
    const Here here;
    const Plan p = plan(here, a[1]);
    const at::Tensor& x = plain(tokens(here, tensor(a[0]), p));
    const float* const weights = weights_of(here, a[2], p);
    const at::Tensor rows = apart(output_as(here, a[4], a[3], x.scalar_type(), {p.rows, x.size(1)}), x);
    at::Tensor other, dots;
    if (a[5] != Py_None) {
        other = contiguous(here, a[5], rows.scalar_type(), {p.rows, x.size(1)});
        dots = here.make({p.T, p.k}, ScalarType::Float);
    }
    run_gather(here, p, x, weights, rows, other, dots);
    return with_dots(a[4], rows, dots);
}

// combine(rows, plan, weights, dtype, y, other)
PyObject* combine(PyObject* const* a) {
    const Here here;
    const Plan p = plan(here, a[1]);
    const at::Tensor& rows = plain(plan_rows(here, tensor(a[0]), p));
    const float* const weights = weights_of(here, a[2], p);
    const at::Tensor y = apart(output_as(here, a[4], a[3], rows.scalar_type(), {p.T, rows.size(1)}), rows);
    at::Tensor other, dots;
    if (a[5] != Py_None) {
        other = tokens(here, tensor(a[5]), p);
        need(other.scalar_type() == y.scalar_type() && other.size(1) == rows.size(1));
        dots = here.make({p.T, p.k}, ScalarType::Float);
    }
    run_combine(here, p, rows, weights, y, other, dots);
    return with_dots(a[4], y, dots);
}

// The gradient of either: the other, with the weights' gradients as dots where they want one.
// A node of the engine's own: its thread takes no interpreter lock for it. 20 tokens of 2 slots,
// 256 columns of bf16, forward and back: gather 27 us, combine with its weights 31; by the classes
// in experts.py 35 and 39 (torch's x * 2: 27).
struct RowsBackward : torch::autograd::Node {
    bool of_gather = false;
    ScalarType type = ScalarType::Float;                    // of the operand
    torch::autograd::SavedVariable weights, other, offsets, row_token, row_of;

    std::string name() const override { return of_gather ? "ExpertsGatherBackward" : "ExpertsCombineBackward"; }
    void release_variables() override {
        const std::lock_guard<std::mutex> lock(mutex_);
        for (torch::autograd::SavedVariable* v : {&weights, &other, &offsets, &row_token, &row_of}) v->reset_data();
    }

    torch::autograd::variable_list apply(torch::autograd::variable_list&& grads) override {
        const std::lock_guard<std::mutex> lock(mutex_);
        torch::autograd::variable_list out(2);
        const bool first = task_should_compute_output(0), second = task_should_compute_output(1);
        if (!grads[0].defined() || !(first || second)) return out;
        const at::Tensor w = weights.unpack(), o = second ? other.unpack() : at::Tensor(), po = offsets.unpack(), pt = row_token.unpack(),
                         pr = row_of.unpack();
        const bool tracked = at::GradMode::is_enabled() &&
                             (grads[0].requires_grad() || (w.defined() && w.requires_grad()) || (o.defined() && o.requires_grad()));
        {
            const at::NoGradGuard no_grad;
            const c10::DeviceGuard device(grads[0].device());
            const Here here;
            try {
                const Plan p = plan(here, po, pt, pr);
                const float* const f = w.defined() ? contiguous(here, w, ScalarType::Float, {p.T, p.k}).const_data_ptr<float>() : nullptr;
                const bool whole_rows = of_gather ? grads[0].is_contiguous() : grads[0].stride(-1) == 1;
                const at::Tensor dy = whole_rows ? grads[0] : grads[0].contiguous();
                if (o.defined()) out[1] = here.make({p.T, p.k}, ScalarType::Float);
                if (of_gather || first) {
                    out[0] = here.make({of_gather ? p.T : p.rows, dy.size(1)}, type);
                    if (of_gather) run_combine(here, p, plan_rows(here, dy, p), f, out[0], o, out[1]);
                    else run_gather(here, p, tokens(here, dy, p), f, out[0], o, out[1]);
                } else {                                    // the dots alone: a combine has them too, beside T rows and not P
                    const at::Tensor unused = here.make({p.T, dy.size(1)}, dy.scalar_type());
                    run_combine(here, p, plan_rows(here, o, p), f, unused, tokens(here, dy, p), out[1]);
                }
                if (!first) out[0].reset();
            } catch (const No&) {
                throw std::runtime_error(name() + ": this gradient cannot be computed");
            }
        }
        if (tracked) {
            for (at::Tensor& t : out)
                if (t.defined()) t.set_requires_grad(true);
            auto twice = std::make_shared<torch::autograd::DelayedError>(name() + " has no gradient of its own", 2);
            out = (*twice)(std::move(out));
        }
        return out;
    }
};

// y, made a function of the operand and the weights for the engine.
PyObject* tracked(const at::Tensor& y, bool of_gather, const at::Tensor& operand, PyObject* weights, PyObject* plan) {
    using torch::autograd::SavedVariable;
    const at::Tensor w = weights == Py_None ? at::Tensor() : tensor(weights);
    auto node = std::shared_ptr<RowsBackward>(new RowsBackward(), torch::autograd::deleteNode);
    node->of_gather = of_gather;
    node->type = operand.scalar_type();
    node->set_next_edges(torch::autograd::collect_next_edges(operand, w));
    node->weights = SavedVariable(w, false);
    if (w.defined() && w.requires_grad()) node->other = SavedVariable(operand, false);
    node->offsets = SavedVariable(tensor(PyTuple_GET_ITEM(plan, 0)), false);
    node->row_token = SavedVariable(tensor(PyTuple_GET_ITEM(plan, 1)), false);
    node->row_of = SavedVariable(tensor(PyTuple_GET_ITEM(plan, 2)), false);
    torch::autograd::set_history(y, node);
    return THPVariable_Wrap(y);
}

const float* tracked_weights(const Here& here, PyObject* o, const Plan& p) {
    if (o == Py_None) return nullptr;
    const at::Tensor& w = contiguous(here, o, ScalarType::Float, {p.T, p.k});
    need(!w._fw_grad(0).defined());
    return w.const_data_ptr<float>();
}

// gather_grad(x, plan, weights)
PyObject* gather_grad(PyObject* const* a) {
    const Here here;
    const Plan p = plan(here, a[1]);
    const at::Tensor& x = tokens(here, tensor(a[0]), p);
    need(at::GradMode::is_enabled() && !x._fw_grad(0).defined());
    const float* const weights = tracked_weights(here, a[2], p);
    const at::Tensor rows = here.make({p.rows, x.size(1)}, x.scalar_type());
    run_gather(here, p, x, weights, rows, at::Tensor(), at::Tensor());
    return tracked(rows, true, x, a[2], a[1]);
}

// combine_grad(rows, plan, weights, dtype)
PyObject* combine_grad(PyObject* const* a) {
    const Here here;
    const Plan p = plan(here, a[1]);
    const at::Tensor& rows = plan_rows(here, tensor(a[0]), p);
    need(at::GradMode::is_enabled() && !rows._fw_grad(0).defined());
    const float* const weights = tracked_weights(here, a[2], p);
    const at::Tensor y = output_as(here, Py_None, a[3], rows.scalar_type(), {p.T, rows.size(1)});
    run_combine(here, p, rows, weights, y, at::Tensor(), at::Tensor());
    return tracked(y, false, rows, a[2], a[1]);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        if (n == N) return F(args);
    } catch (const No&) {
    } catch (const std::exception&) {              // no device, no memory: the long way says so
    }
    PyErr_Clear();                                 // an operand's own error: the long way meets it again
    Py_RETURN_NONE;
}

// types(MX, ExpertPlan): the named tuples of the public interface
PyObject* types(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 2 || !PyType_Check(args[0]) || !PyType_Check(args[1]) ||
        !PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(args[0]), &PyTuple_Type) ||
        !PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(args[1]), &PyTuple_Type)) {
        PyErr_SetString(PyExc_TypeError, "two tuple types are needed");
        return nullptr;
    }
    Py_INCREF(args[0]);
    Py_INCREF(args[1]);
    mx_type = reinterpret_cast<PyTypeObject*>(args[0]);
    plan_type = reinterpret_cast<PyTypeObject*>(args[1]);
    Py_RETURN_NONE;
}

// types_w4(W4)
PyObject* types_w4(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 1 || !PyType_Check(args[0]) || !PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(args[0]), &PyTuple_Type)) {
        PyErr_SetString(PyExc_TypeError, "a tuple type is needed");
        return nullptr;
    }
    Py_INCREF(args[0]);
    w4_type = reinterpret_cast<PyTypeObject*>(args[0]);
    Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"types", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(types)), METH_FASTCALL, nullptr},
    ENTRY(quantize, 2),
    ENTRY(dequantize, 3),
    ENTRY(linear, 5),
    ENTRY(route, 11),
    ENTRY(expert_plan, 2),
    ENTRY(experts_up, 6),
    ENTRY(experts_down, 6),
    {"types_w4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(types_w4)), METH_FASTCALL, nullptr},
    ENTRY(w4_quantize, 5),
    ENTRY(w4_pack, 4),
    ENTRY(w4_dequantize, 3),
    ENTRY(w4_linear, 5),
    ENTRY(w4_experts, 6),
    ENTRY(gather, 6),
    ENTRY(combine, 6),
    ENTRY(gather_grad, 3),
    ENTRY(combine_grad, 4),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "short way to the library's calls", -1, methods};

}  // namespace

// Objects of this Python and this torch are read by their layout in memory, so the module
// does not load with others than it was built for.
PyMODINIT_FUNC PyInit__binding() {
    const char* const python = Py_GetVersion();                       // "major.minor.micro ..."
    const size_t n = sizeof(MQ_PYTHON_VERSION) - 1;
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
    PyObject* text = version ? PyObject_Str(version) : nullptr;
    const char* const now = text ? PyUnicode_AsUTF8(text) : nullptr;
    PyObject* made = nullptr;
    if (now) {
        if (strncmp(python, MQ_PYTHON_VERSION, n) == 0 && strcmp(now, MQ_TORCH_VERSION) == 0) {
            made = PyModule_Create(&module);
        } else {
            PyErr_Format(PyExc_ImportError, "built for Python " MQ_PYTHON_VERSION "x and torch " MQ_TORCH_VERSION ", this is torch %s",
                         now);
        }
    }
    Py_XDECREF(text);
    Py_XDECREF(version);
    Py_XDECREF(torch);
    return made;
}
