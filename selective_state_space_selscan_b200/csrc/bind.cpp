// bind.cpp -- the Python side of the entry points that small calls go through:
// reads pointer, type, shape and strides of torch tensors, picks the tensors'
// device and its current stream, and calls the C ABI (include/selscan.h).
// It does what the ctypes binding does in Python, in a tenth of the time (a
// decode step passes a dozen tensors; marshalling them in Python took longer
// than the kernels).  No arithmetic.
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "selscan.h"

// The torch and the Python that this file is built for (build.py): the package
// looks for it in the file before it loads it.
#ifndef SELSCAN_BIND_STAMP
#error "define SELSCAN_BIND_STAMP"
#endif
extern "C" __attribute__((used, visibility("default"))) const char selscan_bind_stamp[] =
    SELSCAN_BIND_STAMP;

namespace {

struct Args {
    PyObject *const *a;
    Py_ssize_t n;
    Py_ssize_t at = 0;
    int dev = -1;
    bool bad = false;       // a Python error is set
    selscan_tensor d[20];
    int used = 0;

    PyObject *next()
    {
        if (at >= n) {
            if (!bad)
                PyErr_SetString(PyExc_TypeError, "libselscan binding: too few arguments");
            bad = true;
            return nullptr;
        }
        return a[at++];
    }

    // the next argument, a tensor or None
    selscan_tensor *tensor()
    {
        PyObject *o = next();
        if (bad || o == Py_None)
            return nullptr;
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "libselscan takes torch tensors (got %s)",
                         Py_TYPE(o)->tp_name);
            bad = true;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda()) {
            PyErr_Format(PyExc_ValueError,
                         "libselscan takes CUDA tensors only (got one on %s); there is no CPU "
                         "implementation",
                         t.device().str().c_str());
            bad = true;
            return nullptr;
        }
        const int on = t.get_device();
        if (dev >= 0 && on != dev) {
            PyErr_Format(PyExc_ValueError, "tensors on different devices (cuda:%d and cuda:%d)",
                         dev, on);
            bad = true;
            return nullptr;
        }
        dev = on;
        const int64_t nd = t.dim();
        if (nd < 1 || nd > 4) {
            PyErr_Format(PyExc_ValueError,
                         "libselscan takes tensors of 1 to 4 dimensions (got %d)", int(nd));
            bad = true;
            return nullptr;
        }
        selscan_tensor &s = d[used++];
        s.data = t.data_ptr();
        const auto st = t.scalar_type();
        s.dtype = st == at::kFloat      ? SELSCAN_F32
                  : st == at::kBFloat16 ? SELSCAN_BF16
                  : st == at::kInt      ? SELSCAN_I32
                                        : -1;
        s.ndim = int32_t(nd);
        for (int64_t i = 0; i < 4; ++i) {
            s.shape[i] = i < nd ? t.size(i) : 0;
            s.stride[i] = i < nd ? t.stride(i) : 0;
        }
        return &s;
    }

    int64_t integer()
    {
        PyObject *o = next();
        if (bad)
            return 0;
        const long long v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred())
            bad = true;
        return v;
    }
};

enum Entry { kStepSlots, kStepScalarSlots, kFwdPacked, kConv, kConvBwd, kConvStep, kConvPacked };

// call(entry, stream handle or None, the entry point's arguments in order) ->
// status
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    Args a{args, nargs};
    try {
        const int64_t entry = a.integer();
        PyObject *so = a.next();
        if (a.bad)
            return nullptr;
        selscan_tensor *t[20];
        int64_t num[2] = {0, 0};
        // where the numbers stand among the tensors, by entry point
        const auto take = [&](int first, int count) {
            for (int i = first; i < first + count && !a.bad; ++i)
                t[i] = a.tensor();
        };
        switch (entry) {
        case kStepSlots: take(0, 5); num[0] = a.integer(); take(5, 6); break;
        case kStepScalarSlots:
            take(0, 5); num[0] = a.integer(); take(5, 5); num[1] = a.integer(); take(10, 1); break;
        case kFwdPacked: take(0, 4); num[0] = a.integer(); take(4, 9); break;
        case kConv: take(0, 3); num[0] = a.integer(); take(3, 3); break;
        case kConvBwd: take(0, 3); num[0] = a.integer(); take(3, 7); break;
        case kConvStep: take(0, 5); num[0] = a.integer(); take(5, 1); break;
        case kConvPacked: take(0, 4); num[0] = a.integer(); take(4, 4); break;
        default: PyErr_SetString(PyExc_ValueError, "libselscan binding: unknown entry point"); return nullptr;
        }
        if (a.bad)
            return nullptr;
        cudaStream_t s = nullptr;
        const bool given = so != Py_None;
        if (given) {
            s = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(so));
            if (PyErr_Occurred())
                return nullptr;
        }
        c10::cuda::OptionalCUDAGuard guard;
        if (a.dev >= 0) {
            guard.set_index(c10::DeviceIndex(a.dev));
            if (!given)
                s = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(a.dev)).stream();
        }
        selscan_status rc = SELSCAN_OK;
        const int f = int(num[0]);
        Py_BEGIN_ALLOW_THREADS
        switch (entry) {
        case kStepSlots:
            rc = selscan_step_slots(t[0], t[1], t[2], t[3], t[4], f, t[5], t[6], t[7], t[8], t[9],
                                    t[10], s);
            break;
        case kStepScalarSlots:
            rc = selscan_step_scalarA_slots(t[0], t[1], t[2], t[3], t[4], f, t[5], t[6], t[7], t[8],
                                            t[9], num[1], t[10], s);
            break;
        case kFwdPacked:
            rc = selscan_fwd_packed(t[0], t[1], t[2], t[3], f, t[4], t[5], t[6], t[7], t[8], t[9],
                                    t[10], t[11], t[12], s);
            break;
        case kConv:
            rc = selscan_conv(t[0], t[1], t[2], f, t[3], t[4], t[5], s);
            break;
        case kConvBwd:
            rc = selscan_conv_bwd(t[0], t[1], t[2], f, t[3], t[4], t[5], t[6], t[7], t[8], t[9], s);
            break;
        case kConvStep:
            rc = selscan_conv_step(t[0], t[1], t[2], t[3], t[4], f, t[5], s);
            break;
        default:
            rc = selscan_conv_packed(t[0], t[1], t[2], t[3], f, t[4], t[5], t[6], t[7], s);
        }
        Py_END_ALLOW_THREADS
        return PyLong_FromLong(long(rc));
    } catch (const std::exception &e) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// empty(like, fp32, sizes...) -> a contiguous tensor on like's device, of its
// type or fp32
PyObject *empty(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (nargs < 3 || nargs > 6 || !THPVariable_Check(args[0])) {
        PyErr_SetString(PyExc_TypeError, "empty(like, fp32, sizes...)");
        return nullptr;
    }
    try {
        const at::Tensor &like = THPVariable_Unpack(args[0]);
        int64_t size[4];
        for (Py_ssize_t i = 2; i < nargs; ++i) {
            size[i - 2] = PyLong_AsLongLong(args[i]);
            if (size[i - 2] == -1 && PyErr_Occurred())
                return nullptr;
        }
        const auto type = args[1] == Py_True ? at::kFloat : like.scalar_type();
        return THPVariable_Wrap(at::empty(at::IntArrayRef(size, size_t(nargs - 2)),
                                          at::TensorOptions().dtype(type).device(like.device())));
    } catch (const std::exception &e) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyMethodDef methods[] = {
    {"empty", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(empty)), METH_FASTCALL,
     "empty(like, fp32, sizes...) -> tensor"},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL,
     "call(entry, stream handle or None, arguments...) -> status"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "libselscan entry points on torch tensors", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) { return PyModule_Create(&module); }
