// torch_calls.cpp -- the host side of two Python calls in one step: checks, outputs,
// workspace and the call of attn.h.
//
// A small call is bound by what its wrapper does on the host.  Done in Python, one of
// rotary positions takes 13.8 us for a kernel of 2.7: 5.9 for two allocations between
// other work, 1.4 for the foreign-function interface, 4 for checks.  Here the checks that
// an ordinary call passes are made on the tensors themselves.  What does not pass them (an
// error, a tensor on a device that is not the current one, a subclass of Tensor, one whose
// gradient autograd would record) is
// answered with None, and the wrapper goes its own way, which says what is wrong.
//
// bind(address of attn_rotary, of attn_bwd_workspace_size, of attn_bwd): first, once; the
//     functions of the libattn.so that the process uses
// rotary(q, k, pos, transpose, turns, width, interleaved, amplitude, device index of turns)
//     -> (q', k')
// attention_bwd(q, k, v, o, lse, do, dlse, causal, scale) -> (dq, dk, dv)
// or the status of attn.h where it is not ATTN_OK.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <limits.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "attn.h"

namespace {

// what `bind` was given
decltype(&attn_rotary) call_rotary;
decltype(&attn_bwd_workspace_size) call_bwd_workspace_size;
decltype(&attn_bwd) call_bwd;

struct WithoutGil {  // allocations and launches may wait; other threads run meanwhile
    PyThreadState *state = PyEval_SaveThread();
    ~WithoutGil() { PyEval_RestoreThread(state); }
};

const at::Tensor *tensor(PyObject *x) { return THPVariable_CheckExact(x) ? &THPVariable_Unpack(x) : nullptr; }

bool recorded(const at::Tensor *t) { return t && t->requires_grad() && c10::GradMode::is_enabled(); }

bool whole(const at::Tensor &t, at::ScalarType type, c10::Device dev) {
    return t.scalar_type() == type && t.device() == dev && t.is_contiguous();
}

bool fits_int(const at::Tensor &t) {
    for (int64_t n : t.sizes())
        if (n > INT_MAX) return false;
    return true;
}

// attn_dtype of inputs and outputs of these types, or -1
int type_code(at::ScalarType in, at::ScalarType out) {
    if (in == at::kFloat) return out == at::kFloat ? ATTN_F32 : -1;
    if (in == at::kBFloat16) return out == in ? ATTN_BF16 : out == at::kFloat ? ATTN_BF16_OUT_F32 : -1;
    if (in == at::kHalf) return out == in ? ATTN_F16 : out == at::kFloat ? ATTN_F16_OUT_F32 : -1;
    return -1;
}

void *stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

attn_heads heads(const at::Tensor &in, const at::Tensor &out) {
    attn_heads h{};
    h.in = in.data_ptr();
    h.out = out.data_ptr();
    h.H = (int)in.size(1);
    for (int i = 0; i < 3; ++i) {
        h.in_stride[i] = in.stride(i);
        h.out_stride[i] = out.stride(i);
    }
    return h;
}

PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "three addresses expected");
        return nullptr;
    }
    void *at[3];
    for (int i = 0; i < 3; ++i) at[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
    call_rotary = (decltype(call_rotary))at[0];
    call_bwd_workspace_size = (decltype(call_bwd_workspace_size))at[1];
    call_bwd = (decltype(call_bwd))at[2];
    Py_RETURN_NONE;
}

PyObject *rotary(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9 || !call_rotary) Py_RETURN_NONE;
    const at::Tensor *q = tensor(args[0]), *k = args[1] == Py_None ? nullptr : tensor(args[1]), *pos = tensor(args[2]);
    if (!q || !pos || (!k && args[1] != Py_None) || q->dim() != 4 || !q->is_cuda() ||
        recorded(q) || recorded(k))
        Py_RETURN_NONE;
    const c10::Device dev = q->device();
    const int64_t B = q->size(0), S = q->size(2), d = q->size(3);
    const int code = type_code(q->scalar_type(), q->scalar_type());
    if (code < 0 || dev.index() != c10::cuda::current_device() || !fits_int(*q) || q->stride(3) != 1) Py_RETURN_NONE;
    if (k && (k->dim() != 4 || k->scalar_type() != q->scalar_type() || k->device() != dev || k->size(0) != B ||
              k->size(2) != S || k->size(3) != d || !fits_int(*k) || k->stride(3) != 1))
        Py_RETURN_NONE;
    const bool per_token = pos->dim() == 2;
    if (!whole(*pos, at::kInt, dev) || (pos->dim() != 1 && !per_token) || pos->size(0) != B ||
        (per_token && pos->size(1) != S))
        Py_RETURN_NONE;
    const int transpose = PyObject_IsTrue(args[3]);
    const auto *turns = (const uint64_t *)PyLong_AsVoidPtr(args[4]);
    const long width = PyLong_AsLong(args[5]), interleaved = PyLong_AsLong(args[6]);
    const double amplitude = PyFloat_AsDouble(args[7]);
    const long turns_on = PyLong_AsLong(args[8]);  // -1: the host
    if (PyErr_Occurred()) return nullptr;
    if (width > d || turns_on != dev.index()) Py_RETURN_NONE;
    int st;
    at::Tensor qo, ko;
    {
        WithoutGil free;
        qo = at::empty(q->sizes(), q->options());
        if (k) ko = at::empty(k->sizes(), k->options());
        const attn_heads hq = heads(*q, qo), hk = k ? heads(*k, ko) : attn_heads{};
        st = call_rotary(&hq, k ? &hk : nullptr, turns, (int)width, (int)interleaved, (float)amplitude, transpose,
                         (const int32_t *)pos->data_ptr(), per_token, (int)B, (int)S, (int)d, code, stream_of(dev));
    }
    if (st != ATTN_OK) return PyLong_FromLong(st);
    PyObject *a = THPVariable_Wrap(qo), *b = k ? THPVariable_Wrap(ko) : Py_NewRef(Py_None);
    return a && b ? Py_BuildValue("(NN)", a, b) : nullptr;
    END_HANDLE_TH_ERRORS
}

PyObject *attention_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9 || !call_bwd || !call_bwd_workspace_size) Py_RETURN_NONE;
    const at::Tensor *t[7];  // q, k, v, o, lse, do, dlse
    for (int i = 0; i < 7; ++i) {
        t[i] = args[i] == Py_None && i == 6 ? nullptr : tensor(args[i]);
        if ((!t[i] && !(args[i] == Py_None && i == 6)) || recorded(t[i])) Py_RETURN_NONE;
    }
    const at::Tensor &q = *t[0], &k = *t[1], &v = *t[2], &o = *t[3], &lse = *t[4], &dout = *t[5];
    if (q.dim() != 4 || k.dim() != 4 || !q.is_cuda()) Py_RETURN_NONE;
    const c10::Device dev = q.device();
    const at::ScalarType in = q.scalar_type(), out = o.scalar_type();
    const int code = type_code(in, out);
    const int64_t B = q.size(0), H = q.size(1), Sq = q.size(2), d = q.size(3), H_kv = k.size(1), Skv = k.size(2);
    if (code < 0 || dev.index() != c10::cuda::current_device() || !fits_int(q) || !fits_int(k) || H < 1 || H_kv < 1 ||
        H % H_kv != 0 || k.size(0) != B || k.size(3) != d || v.sizes() != k.sizes() || o.sizes() != q.sizes() ||
        dout.sizes() != q.sizes())
        Py_RETURN_NONE;
    if (!whole(q, in, dev) || !whole(k, in, dev) || !whole(v, in, dev) || !whole(dout, in, dev) || !whole(o, out, dev))
        Py_RETURN_NONE;
    for (const at::Tensor *x : {t[4], t[6]})
        if (x && (!whole(*x, at::kFloat, dev) || x->sizes() != q.sizes().slice(0, 3))) Py_RETURN_NONE;
    const int causal = PyObject_IsTrue(args[7]);
    const double scale = PyFloat_AsDouble(args[8]);
    if (PyErr_Occurred()) return nullptr;
    int st;
    at::Tensor dq, dk, dv;
    {
        WithoutGil free;
        size_t need = 0;
        st = call_bwd_workspace_size((int)B, (int)H, (int)H_kv, (int)Sq, (int)Skv, (int)d, causal, code, &need);
        if (st == ATTN_OK) {
            const auto like = q.options().dtype(out);
            dq = at::empty(q.sizes(), like);
            dk = at::empty(k.sizes(), like);
            dv = at::empty(k.sizes(), like);
            // returned to the allocator behind the launch, for later work on this stream
            at::Tensor work;
            if (need) work = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
            st = call_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), (const float *)lse.data_ptr(),
                          dout.data_ptr(), t[6] ? (const float *)t[6]->data_ptr() : nullptr, dq.data_ptr(),
                          dk.data_ptr(), dv.data_ptr(), (int)B, (int)H, (int)H_kv, (int)Sq, (int)Skv, (int)d, causal,
                          (float)scale, code, need ? work.data_ptr() : nullptr, need, stream_of(dev));
        }
    }
    if (st != ATTN_OK) return PyLong_FromLong(st);
    PyObject *a = THPVariable_Wrap(dq), *b = THPVariable_Wrap(dk), *c = THPVariable_Wrap(dv);
    return a && b && c ? Py_BuildValue("(NNN)", a, b, c) : nullptr;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {{"bind", (PyCFunction)(void (*)())bind, METH_FASTCALL, nullptr},
                         {"rotary", (PyCFunction)(void (*)())rotary, METH_FASTCALL, nullptr},
                         {"attention_bwd", (PyCFunction)(void (*)())attention_bwd, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
