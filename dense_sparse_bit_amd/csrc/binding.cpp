// The short way from Python to the microscaled and routing calls (include/mq.h).
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
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string.h>

#include "../../include/mq.h"

#define MQ_TEXT_(x) #x
#define MQ_TEXT(x) MQ_TEXT_(x)
#define MQ_PYTHON_VERSION MQ_TEXT(PY_MAJOR_VERSION) "." MQ_TEXT(PY_MINOR_VERSION) "."

namespace {

using at::ScalarType;

PyTypeObject* mx_type = nullptr;
PyTypeObject* plan_type = nullptr;

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

const at::Tensor& contiguous(const Here& here, PyObject* o, ScalarType type, at::IntArrayRef size) {
    const at::Tensor& t = tensor(o);
    need(t.scalar_type() == type && t.sizes() == size && here.has(t) && t.is_contiguous());
    return t;
}

// a strided matrix whose last axis is contiguous
const at::Tensor& input(const Here& here, PyObject* o, int64_t dims) {
    const at::Tensor& t = tensor(o);
    need(t.dim() == dims && here.has(t) && (t.stride(-1) == 1 || t.size(-1) <= 1));
    return t;
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

PyObject* wrapped(PyObject* given, const at::Tensor& y) {
    if (given == Py_None) return THPVariable_Wrap(y);
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

Plan plan(const Here& here, PyObject* o) {
    need(whole(o, plan_type, 3));
    const at::Tensor &offsets = tensor(PyTuple_GET_ITEM(o, 0)), &row_of = tensor(PyTuple_GET_ITEM(o, 2));
    need(row_of.dim() == 2 && offsets.dim() == 1);
    Plan p;
    p.T = row_of.size(0);
    p.k = row_of.size(1);
    p.E = offsets.size(0) - 1;
    p.rows = mq_plan_rows(p.T, p.k, p.E);
    need(p.rows >= 0);
    p.offsets = contiguous(here, PyTuple_GET_ITEM(o, 0), ScalarType::Int, {p.E + 1}).const_data_ptr<int32_t>();
    p.row_token = contiguous(here, PyTuple_GET_ITEM(o, 1), ScalarType::Int, {p.rows}).const_data_ptr<int32_t>();
    p.row_of = contiguous(here, PyTuple_GET_ITEM(o, 2), ScalarType::Int, {p.T, p.k}).const_data_ptr<int32_t>();
    return p;
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
