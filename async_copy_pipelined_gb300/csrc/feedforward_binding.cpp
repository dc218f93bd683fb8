// The ordinary calls of the feed-forward operators, from Python to the C ABI.
//
// A call with a handful of tensors takes the interpreter about 10 us of checks,
// allocations and marshalling next to 4 us of launch; here it takes 1.5 (a
// quantisation 14.8 and 4.6 us in all).  What is ordinary: strided tensors on the
// current device, results allocated by the call, the current stream.  Everything
// else (other streams, given results, empty operands, anything to refuse, a status
// that is not GEMM_OK) returns None, and feedforward.py does the call or raises
// its error.
//
// The interpreter's lock is let go while results are allocated and kernels
// enqueued, as both may wait for the device.
//
// It takes the addresses of the library's functions from feedforward.py and uses
// torch for tensors alone.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstring>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pipelined_ffn.h"

namespace {

decltype(&::gated_projection) entry_gated;
decltype(&::gated_projection_backward) entry_gated_backward;
decltype(&::gated_projection_backward_workspace) entry_gated_backward_workspace;
decltype(&::quantize_fp8) entry_quantize;
decltype(&::gemm_fp8) entry_gemm;

constexpr int64_t kMaxSide = int64_t{1} << 30;
constexpr int64_t kBlock = 128;

int64_t up_to(int64_t n, int64_t step) { return (n + step - 1) / step * step; }

// A tensor's matrix, its rows' elements side by side.
struct Matrix {
    void *p;
    int64_t rows, cols, pitch;
};

const at::Tensor *tensor(PyObject *o)
{
    // Not of subclasses, which may not have memory to point at.
    return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

bool on(const at::Tensor &t, int device) { return t.is_cuda() && t.get_device() == device; }

bool sides(const at::Tensor &t)
{
    return t.dim() == 2 && t.size(0) >= 1 && t.size(1) >= 1 && t.size(0) <= kMaxSide && t.size(1) <= kMaxSide;
}

bool matrix(const at::Tensor *t, at::ScalarType type, int device, Matrix *m)
{
    if (!t || !on(*t, device) || t->scalar_type() != type || !sides(*t) || t->stride(1) != 1)
        return false;
    *m = Matrix{t->data_ptr(), t->size(0), t->size(1), t->size(0) > 1 ? t->stride(0) : t->size(1)};
    return m->pitch >= m->cols;
}

// A bfloat16 tensor as rows of its last dimension, at one common distance.
bool tokens(const at::Tensor *t, int device, Matrix *m)
{
    if (!t || !on(*t, device) || t->scalar_type() != at::kBFloat16)
        return false;
    const auto size = t->sizes(), stride = t->strides();
    const int64_t last = static_cast<int64_t>(size.size()) - 1;
    if (last < 0 || size[last] < 1 || size[last] > kMaxSide || stride[last] != 1)
        return false;
    int64_t rows = 1, pitch = size[last];
    for (int64_t i = last - 1; i >= 0; --i) {
        if (size[i] == 1)
            continue;
        if (rows == 1)
            pitch = stride[i];
        else if (stride[i] != pitch * rows)
            return false;
        // At most kMaxSide squared: no overflow.
        if (size[i] < 1 || size[i] > kMaxSide || (rows *= size[i]) > kMaxSide)
            return false;
    }
    *m = Matrix{t->data_ptr(), rows, size[last], pitch};
    return pitch >= size[last];
}

// Without the interpreter's lock.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// The current device's index where x is on it, else -1.
int device_of(const at::Tensor *x)
{
    if (!x || !x->is_cuda())
        return -1;
    const int device = x->get_device();
    return c10::cuda::current_device() == device ? device : -1;
}

void *stream_of(int device) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }

// feedforward.py's _pitch and _new_rows.
int64_t pitch_of(int64_t cols, int64_t step) { return cols % step == 0 ? cols : up_to(cols, 2 * step); }

at::Tensor new_rows(at::IntArrayRef size, int64_t step, const at::TensorOptions &options)
{
    const int64_t pitch = pitch_of(size.back(), step);
    if (pitch == size.back())
        return at::empty(size, options);
    c10::SmallVector<int64_t, 5> stride(size.size(), 1);
    int64_t distance = pitch;
    for (size_t i = size.size() - 1; i-- > 0; distance *= size[i])
        stride[i] = distance;
    return at::empty_strided(size, stride, options);
}

at::Tensor new_rows(int64_t rows, int64_t cols, int64_t step, const at::TensorOptions &options)
{
    const int64_t size[2] = {rows, cols};
    return new_rows(at::IntArrayRef(size, 2), step, options);
}

PyObject *wrap(at::Tensor t) { return t.defined() ? THPVariable_Wrap(std::move(t)) : Py_NewRef(Py_None); }

PyObject *three(at::Tensor a, at::Tensor b, at::Tensor c)
{
    PyObject *t = PyTuple_New(3);
    if (!t)
        return nullptr;
    PyTuple_SET_ITEM(t, 0, wrap(std::move(a)));
    PyTuple_SET_ITEM(t, 1, wrap(std::move(b)));
    PyTuple_SET_ITEM(t, 2, wrap(std::move(c)));
    return t;
}

PyObject *none() { return Py_NewRef(Py_None); }

// (x, w_gate, w_up, activation, save)
PyObject *gated_projection_py(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 5)
        return none();
    const at::Tensor *x = tensor(args[0]);
    const int device = device_of(x);
    Matrix mx, mg, mu;
    if (device < 0 || !tokens(x, device, &mx) ||
        !matrix(tensor(args[1]), at::kBFloat16, device, &mg) || !matrix(tensor(args[2]), at::kBFloat16, device, &mu) ||
        mg.rows != mx.cols || mu.rows != mx.cols || mu.cols != mg.cols)
        return none();
    const long activation = PyLong_AsLong(args[3]);
    const int save = PyObject_IsTrue(args[4]);
    if (save < 0)
        return none();
    const auto options = x->options().requires_grad(false);
    const int64_t hidden = mg.cols, pitch = pitch_of(hidden, 8);
    c10::SmallVector<int64_t, 5> size(x->sizes().begin(), x->sizes().end());
    size.back() = hidden;
    at::Tensor h, gate, up;
    int status;
    {
        Unlocked unlocked;
        h = new_rows(size, 8, options);
        if (save) {
            gate = new_rows(size, 8, options);
            up = new_rows(size, 8, options);
        }
        status = entry_gated(static_cast<int>(mx.rows), static_cast<int>(mx.cols), static_cast<int>(hidden), mx.p,
                             mx.pitch, mg.p, mg.pitch, mu.p, mu.pitch, h.data_ptr(), pitch,
                             save ? gate.data_ptr() : nullptr, pitch, save ? up.data_ptr() : nullptr, pitch,
                             static_cast<int>(activation), stream_of(device));
    }
    if (status != GEMM_OK)
        return none();
    return save ? three(std::move(h), std::move(gate), std::move(up)) : wrap(std::move(h));
}

// Bytes of the gradient's workspace, remembered for the sizes asked for last.
size_t workspace_bytes(int device, int rows, int width, int hidden)
{
    struct Last {
        int device = -1, rows = 0, width = 0, hidden = 0;
        size_t bytes = 0;
    };
    thread_local Last last;
    if (last.device != device || last.rows != rows || last.width != width || last.hidden != hidden) {
        size_t bytes = 0;
        if (entry_gated_backward_workspace(rows, width, hidden, &bytes) != GEMM_OK)
            return 0;
        last = Last{device, rows, width, hidden, bytes};
    }
    return last.bytes;
}

// (dh, x, w_gate, w_up, gate, up, activation, input_grad, weight_grad)
PyObject *gated_projection_backward_py(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 9)
        return none();
    const at::Tensor *x = tensor(args[1]);
    const int device = device_of(x);
    const at::Tensor *over[3] = {tensor(args[0]), tensor(args[4]), tensor(args[5])}; // dh, gate, up
    Matrix mx, mg, mu, mover[3];
    if (device < 0 || !tokens(x, device, &mx) || !matrix(tensor(args[2]), at::kBFloat16, device, &mg) ||
        !matrix(tensor(args[3]), at::kBFloat16, device, &mu))
        return none();
    const int64_t width = mx.cols, hidden = mg.cols;
    if (mg.rows != width || mu.rows != width || mu.cols != hidden)
        return none();
    for (int i = 0; i < 3; ++i)
        if (!tokens(over[i], device, &mover[i]) || mover[i].cols != hidden ||
            over[i]->sizes().slice(0, over[i]->dim() - 1) != x->sizes().slice(0, x->dim() - 1))
            return none();
    const long activation = PyLong_AsLong(args[6]);
    const int input = PyObject_IsTrue(args[7]), weight = PyObject_IsTrue(args[8]);
    if (input < 0 || weight < 0)
        return none();
    const auto options = x->options().requires_grad(false);
    at::Tensor dx, dwg, dwu;
    int status;
    {
        Unlocked unlocked;
        const size_t bytes = workspace_bytes(device, static_cast<int>(mx.rows), static_cast<int>(width),
                                             static_cast<int>(hidden));
        if (input)
            dx = new_rows(x->sizes(), 8, options);
        if (weight) {
            dwg = new_rows(width, hidden, 8, options);
            dwu = new_rows(width, hidden, 8, options);
        }
        at::Tensor workspace = at::empty({static_cast<int64_t>(bytes)}, options.dtype(at::kByte));
        status = entry_gated_backward(
            static_cast<int>(mx.rows), static_cast<int>(width), static_cast<int>(hidden), mover[0].p, mover[0].pitch,
            mx.p, mx.pitch, mg.p, mg.pitch, mu.p, mu.pitch, mover[1].p, mover[1].pitch, mover[2].p, mover[2].pitch,
            input ? dx.data_ptr() : nullptr, pitch_of(width, 8), weight ? dwg.data_ptr() : nullptr, pitch_of(hidden, 8),
            weight ? dwu.data_ptr() : nullptr, pitch_of(hidden, 8), static_cast<int>(activation), workspace.data_ptr(),
            bytes, stream_of(device));
    }
    if (status != GEMM_OK)
        return none();
    return three(std::move(dx), std::move(dwg), std::move(dwu));
}

bool fp8(at::ScalarType t) { return t == at::kFloat8_e4m3fn || t == at::kFloat8_e5m2; }
int format_of(at::ScalarType t) { return t == at::kFloat8_e5m2 ? GEMM_FP8_E5M2 : GEMM_FP8_E4M3; }

// (x, group, format)
PyObject *quantize_fp8_py(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 3)
        return none();
    const at::Tensor *x = tensor(args[0]);
    const int device = device_of(x);
    Matrix m;
    if (device < 0 || (x->scalar_type() != at::kFloat && x->scalar_type() != at::kBFloat16) ||
        !matrix(x, x->scalar_type(), device, &m))
        return none();
    const long group = PyLong_AsLong(args[1]), format = PyLong_AsLong(args[2]);
    if (group < GEMM_FP8_ROW || group > GEMM_FP8_BLOCK || (format != GEMM_FP8_E4M3 && format != GEMM_FP8_E5M2))
        return none();
    const auto options = x->options().requires_grad(false);
    const int64_t scale_rows = group == GEMM_FP8_ROW ? m.rows : (m.rows + kBlock - 1) / kBlock;
    const int64_t scale_cols = group == GEMM_FP8_COLUMN ? m.cols : (m.cols + kBlock - 1) / kBlock;
    at::Tensor q, scale;
    int status;
    {
        Unlocked unlocked;
        q = new_rows(m.rows, m.cols, 16,
                     options.dtype(format == GEMM_FP8_E5M2 ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn));
        scale = at::empty({scale_rows, scale_cols}, options.dtype(at::kFloat));
        status = entry_quantize(static_cast<int>(m.rows), static_cast<int>(m.cols), m.p, m.pitch,
                                x->scalar_type() == at::kFloat ? GEMM_DTYPE_F32 : GEMM_DTYPE_BF16,
                                static_cast<int>(group), static_cast<int>(format), q.data_ptr(), pitch_of(m.cols, 16),
                                static_cast<float *>(scale.data_ptr()), scale_cols, stream_of(device));
    }
    if (status != GEMM_OK)
        return none();
    PyObject *t = PyTuple_New(2);
    if (!t)
        return nullptr;
    PyTuple_SET_ITEM(t, 0, wrap(std::move(q)));
    PyTuple_SET_ITEM(t, 1, wrap(std::move(scale)));
    return t;
}

// An 8-bit operand, its rows or its columns side by side.
struct Operand {
    void *p;
    int64_t rows, cols, pitch;
    int format, transposed;
};

bool operand(const at::Tensor *t, int device, Operand *o)
{
    if (!t || !on(*t, device) || !fp8(t->scalar_type()) || !sides(*t))
        return false;
    const int64_t rows = t->size(0), cols = t->size(1), sr = t->stride(0), sc = t->stride(1);
    *o = Operand{t->data_ptr(), rows, cols, 0, format_of(t->scalar_type()), 0};
    if (cols == 1 && rows > 1 && sr == 1) { // one row's transpose
        o->pitch = up_to(rows, 16);
        o->transposed = 1;
    } else if ((cols == 1 || sc == 1) && (rows == 1 || sr >= cols)) {
        o->pitch = rows > 1 ? sr : up_to(cols, 16);
    } else if ((rows == 1 || sr == 1) && (cols == 1 || sc >= rows)) {
        o->pitch = cols > 1 ? sc : up_to(rows, 16);
        o->transposed = 1;
    } else {
        return false;
    }
    return true;
}

struct Scales {
    const float *p;
    int64_t side, block; // strides along the rows or columns, and along K
    int group;
};

// Scales of `sides` rows (columns: along 1) and `blocks` blocks.
bool scales(const at::Tensor *t, int device, int64_t sides, int64_t blocks, int along, Scales *s)
{
    if (!t || !on(*t, device) || t->scalar_type() != at::kFloat || t->dim() != 2 || t->size(1 - along) != blocks)
        return false;
    const int64_t given = t->size(along);
    if (given != sides && given != (sides + kBlock - 1) / kBlock)
        return false;
    *s = Scales{static_cast<const float *>(t->data_ptr()), t->stride(along), t->stride(1 - along),
                given == sides ? 1 : static_cast<int>(kBlock)};
    return true;
}

// (A, B, a_scale, b_scale, dtype)
PyObject *gemm_fp8_py(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 5)
        return none();
    const at::Tensor *ta = tensor(args[0]);
    const int device = device_of(ta);
    Operand a, b;
    if (device < 0 || !operand(ta, device, &a) || !operand(tensor(args[1]), device, &b) || a.cols != b.rows)
        return none();
    const int64_t blocks = (a.cols + kBlock - 1) / kBlock;
    Scales sa, sb;
    if (!scales(tensor(args[2]), device, a.rows, blocks, 0, &sa) ||
        !scales(tensor(args[3]), device, b.cols, blocks, 1, &sb))
        return none();
    const long dtype = PyLong_AsLong(args[4]);
    if (dtype != GEMM_DTYPE_F32 && dtype != GEMM_DTYPE_BF16)
        return none();
    const int64_t step = dtype == GEMM_DTYPE_F32 ? 4 : 8; // rows at multiples of 16 bytes
    at::Tensor c;
    int status;
    {
        Unlocked unlocked;
        c = new_rows(a.rows, b.cols, step, ta->options().requires_grad(false).dtype(
                                               dtype == GEMM_DTYPE_F32 ? at::kFloat : at::kBFloat16));
        status = entry_gemm(static_cast<int>(a.rows), static_cast<int>(b.cols), static_cast<int>(a.cols), a.p, a.pitch,
                            a.format, a.transposed, sa.p, sa.side, sa.block, sa.group, b.p, b.pitch, b.format,
                            b.transposed, sb.p, sb.block, sb.side, sb.group, c.data_ptr(),
                            pitch_of(b.cols, step),
                            static_cast<int>(dtype), stream_of(device));
    }
    if (status != GEMM_OK)
        return none();
    return wrap(std::move(c));
}

// A C++ exception (no memory for a result) ends here: feedforward.py makes the
// call again and raises what it comes to.  Integers that were none leave no error.
template <PyObject *(*Call)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    PyObject *r = nullptr;
    try {
        r = Call(self, args, n);
    } catch (...) {
        r = none();
    }
    if (r == Py_None)
        PyErr_Clear();
    return r;
}

// (addresses of the five functions)
PyObject *entries(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "five addresses");
        return nullptr;
    }
    void *p[5];
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (!p[i]) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    entry_gated = reinterpret_cast<decltype(entry_gated)>(p[0]);
    entry_gated_backward = reinterpret_cast<decltype(entry_gated_backward)>(p[1]);
    entry_gated_backward_workspace = reinterpret_cast<decltype(entry_gated_backward_workspace)>(p[2]);
    entry_quantize = reinterpret_cast<decltype(entry_quantize)>(p[3]);
    entry_gemm = reinterpret_cast<decltype(entry_gemm)>(p[4]);
    return none();
}

template <class F>
PyCFunction fast(F f)
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"entries", fast(entries), METH_FASTCALL, nullptr},
    {"gated_projection", fast(guarded<gated_projection_py>), METH_FASTCALL, nullptr},
    {"gated_projection_backward", fast(guarded<gated_projection_backward_py>), METH_FASTCALL, nullptr},
    {"quantize_fp8", fast(guarded<quantize_fp8_py>), METH_FASTCALL, nullptr},
    {"gemm_fp8", fast(guarded<gemm_fp8_py>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_feedforward", nullptr, -1, methods,
                      nullptr,               nullptr,        nullptr, nullptr};

} // namespace

// BINDING_TORCH: the whole version of the torch whose headers these are, which its
// own macro cuts to three numbers, the same for several builds.
PyMODINIT_FUNC PyInit__feedforward()
{
    static const char build[] = BINDING_TORCH;
    const std::string version(build, std::strcspn(build, "+"));
    PyObject *m = PyModule_Create(&module);
    if (m && (PyModule_AddStringConstant(m, "torch_build", build) < 0 ||
              PyModule_AddStringConstant(m, "torch_version", version.c_str()) < 0))
        Py_CLEAR(m);
    return m;
}
