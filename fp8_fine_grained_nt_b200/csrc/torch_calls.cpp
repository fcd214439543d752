// The common calls of the grouped operators without Python's cost per tensor:
// operators of a few microseconds would wait for the checks of their arguments
// (adapters for one token: 23 us of the host's time a call through binding.py, 6
// here).
//
// Each function takes the tensors of one call on the current device and
// stream, makes the same checks as its counterpart in binding.py, and calls the
// C ABI.  It returns the call's dg_status, or -1 where a check fails or the
// call is not the common one; binding.py then makes its own checks, which say
// what is wrong, or the call.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fp8_nt.h"

namespace {

constexpr long long kNotHere = -1;

// A call's tensors: every one checked against the device of the first.
struct Call {
    bool ok = true;
    int device = -1;

    const at::Tensor *any(PyObject *o, int ndim)
    {
        if (!ok || !THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.dim() != ndim || t.layout() != at::kStrided) {
            ok = false;
            return nullptr;
        }
        if (device < 0)
            device = t.get_device();
        if (t.get_device() != device) {
            ok = false;
            return nullptr;
        }
        return &t;
    }

    const at::Tensor *dense(PyObject *o, int ndim, at::ScalarType type)
    {
        const at::Tensor *t = any(o, ndim);
        if (t && (t->scalar_type() != type || !t->is_contiguous()))
            ok = false;
        return ok ? t : nullptr;
    }

    // a matrix with contiguous rows
    const at::Tensor *rows(PyObject *o, at::ScalarType type)
    {
        const at::Tensor *t = any(o, 2);
        if (t && (t->scalar_type() != type || (!t->is_contiguous() && t->size(1) != 1 && t->stride(1) != 1)))
            ok = false;
        return ok ? t : nullptr;
    }

    bool here() const { return ok && device == c10::cuda::current_device(); }
    dg_stream_t stream() const { return reinterpret_cast<dg_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream()); }
};

int half_code(const at::Tensor &t)
{
    return t.scalar_type() == at::kBFloat16 ? DG_INPUT_BF16 : t.scalar_type() == at::kHalf ? DG_INPUT_F16 : -1;
}

bool fits(int64_t n) { return n >= 0 && n <= 0x7fffffff; }

// (a, b, d, offsets) of the forward and of the input gradient
template <bool NN>
long long ragged_rows(PyObject *const *args)
{
    Call call;
    const at::Tensor *a = call.any(args[0], 2);
    if (!a || half_code(*a) < 0 || !a->is_contiguous())
        return kNotHere;
    const at::Tensor *b = call.dense(args[1], 3, a->scalar_type()), *d = call.dense(args[2], 2, a->scalar_type()),
                     *offsets = call.dense(args[3], 1, at::kInt);
    if (!call.here())
        return kNotHere;
    const int64_t T = a->size(0), G = b->size(0), N = b->size(1), K = b->size(2);
    if (a->size(1) != (NN ? N : K) || d->size(0) != T || d->size(1) != (NN ? K : N) || offsets->size(0) != G + 1 ||
        !fits(T) || !fits(G) || !fits(N) || !fits(K))
        return kNotHere;
    return (NN ? m_grouped_gemm_nn_ragged : m_grouped_gemm_nt_ragged)(
        a->data_ptr(), b->data_ptr(), d->data_ptr(), static_cast<const int *>(offsets->data_ptr()), half_code(*a),
        (int)G, (int)T, (int)N, (int)K, call.stream());
}

// (a, b, d, offsets, accumulate)
long long ragged_weights(PyObject *const *args)
{
    Call call;
    const at::Tensor *a = call.any(args[0], 2);
    if (!a || half_code(*a) < 0 || !a->is_contiguous())
        return kNotHere;
    const int accumulate = PyObject_IsTrue(args[4]);
    const at::Tensor *b = call.dense(args[1], 2, a->scalar_type()), *d = call.any(args[2], 3),
                     *offsets = call.dense(args[3], 1, at::kInt);
    if (!call.here() || accumulate < 0 || !d->is_contiguous())
        return kNotHere;
    const bool f32 = d->scalar_type() == at::kFloat;
    const int64_t T = a->size(0), G = d->size(0), N = d->size(1), K = d->size(2);
    if ((!f32 && (accumulate || d->scalar_type() != a->scalar_type())) || a->size(1) != N || b->size(0) != T ||
        b->size(1) != K || offsets->size(0) != G + 1 || !fits(T) || !fits(G) || !fits(N) || !fits(K))
        return kNotHere;
    return k_grouped_gemm_tn_ragged(a->data_ptr(), b->data_ptr(), d->data_ptr(),
                                    static_cast<const int *>(offsets->data_ptr()), half_code(*a),
                                    f32 ? DG_INPUT_F32 : half_code(*a), accumulate, (int)G, (int)T, (int)N, (int)K,
                                    call.stream());
}

// (index, num_groups, offsets, order, slots or None, m_indices or None, alignment)
long long group_rows(PyObject *const *args)
{
    Call call;
    const at::Tensor *index = call.any(args[0], 1);
    if (!index || !index->is_contiguous() || !PyLong_Check(args[1]) || !PyLong_Check(args[6]))
        return kNotHere;
    const bool i64 = index->scalar_type() == at::kLong;
    if (!i64 && index->scalar_type() != at::kInt)
        return kNotHere;
    const long groups = PyLong_AsLong(args[1]), alignment = PyLong_AsLong(args[6]);
    const at::Tensor *offsets = call.dense(args[2], 1, at::kInt), *order = call.dense(args[3], 1, at::kInt);
    const at::Tensor *slots = args[4] == Py_None ? nullptr : call.dense(args[4], 1, at::kInt);
    const at::Tensor *m_indices = args[5] == Py_None ? nullptr : call.dense(args[5], 1, at::kInt);
    if (PyErr_Occurred()) {
        PyErr_Clear(); // a count beyond a long
        return kNotHere;
    }
    const int64_t R = index->size(0);
    if (!call.here() || !fits(R) || !fits(groups) || !fits(alignment))
        return kNotHere;
    const int capacity = get_row_groups_capacity((int)R, (int)groups, (int)alignment);
    const long long need = get_group_rows_workspace_size((int)R, (int)groups);
    if (capacity < 0 || need < 0 || offsets->size(0) != groups + 1 || order->size(0) != capacity ||
        (slots && slots->size(0) != R) || (m_indices && m_indices->size(0) != capacity))
        return kNotHere;
    at::Tensor workspace;
    if (need > 0)
        workspace = at::empty({(int64_t)need}, index->options().dtype(at::kByte));
    return group_rows_by_index(index->data_ptr(), i64 ? DG_INDEX_I64 : DG_INDEX_I32,
                               static_cast<int *>(offsets->data_ptr()), static_cast<int *>(order->data_ptr()),
                               slots ? static_cast<int *>(slots->data_ptr()) : nullptr,
                               m_indices ? static_cast<int *>(m_indices->data_ptr()) : nullptr, (int)R, (int)groups,
                               (int)alignment, need > 0 ? workspace.data_ptr() : nullptr, (size_t)need, call.stream());
}

// (x, lora_a, lora_b, scales, c, d, m_indices, order or None)
long long lora_add(PyObject *const *args)
{
    Call call;
    const at::Tensor *x = call.any(args[0], 2);
    if (!x || half_code(*x) < 0)
        return kNotHere;
    const at::ScalarType type = x->scalar_type();
    x = call.rows(args[0], type);
    const at::Tensor *a = call.dense(args[1], 3, type), *b = call.dense(args[2], 3, type),
                     *scales = call.dense(args[3], 1, at::kFloat), *c = call.rows(args[4], type),
                     *d = call.rows(args[5], type), *m_indices = call.dense(args[6], 1, at::kInt);
    const at::Tensor *order = args[7] == Py_None ? nullptr : call.dense(args[7], 1, at::kInt);
    if (!call.here())
        return kNotHere;
    const int64_t L = a->size(0), R = a->size(1), K = a->size(2), T = d->size(0), N = d->size(1), S = m_indices->size(0);
    if (x->size(0) != T || x->size(1) != K || b->size(0) != L || b->size(1) != N || b->size(2) != R ||
        c->size(0) != T || c->size(1) != N || scales->size(0) != L || (order ? order->size(0) != S : S > T) ||
        !fits(L) || !fits(R) || !fits(K) || !fits(T) || !fits(N) || !fits(S))
        return kNotHere;
    const long long need = get_lora_workspace_size((int)S, (int)L, (int)R, (int)N, (int)K);
    if (need < 0)
        return kNotHere;
    at::Tensor workspace;
    if (need > 0)
        workspace = at::empty({(int64_t)need}, x->options().dtype(at::kByte));
    return m_grouped_lora_add(x->data_ptr(), T > 1 ? x->stride(0) : K, a->data_ptr(), b->data_ptr(),
                              static_cast<const float *>(scales->data_ptr()), c->data_ptr(),
                              T > 1 ? c->stride(0) : N, d->data_ptr(), T > 1 ? d->stride(0) : N,
                              static_cast<const int *>(m_indices->data_ptr()),
                              order ? static_cast<const int *>(order->data_ptr()) : nullptr, half_code(*x), (int)S,
                              (int)T, (int)L, (int)R, (int)N, (int)K, need > 0 ? workspace.data_ptr() : nullptr,
                              (size_t)need, call.stream());
}

template <long long (*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    // (C++ exceptions become torch's own in Python: no memory for the workspace is
    // its OutOfMemoryError, as from binding.py)
    HANDLE_TH_ERRORS
    if (n != N)
        return PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    const long long status = F(args);
    return PyErr_Occurred() ? nullptr : PyLong_FromLongLong(status); // (an argument's own error)
    END_HANDLE_TH_ERRORS
}

#define FP8NT_ENTRY(name, f, n)                                                                                       \
    {                                                                                                                 \
        name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f, n>)), METH_FASTCALL, nullptr        \
    }

PyMethodDef kMethods[] = {
    FP8NT_ENTRY("m_grouped_gemm_nt_ragged", ragged_rows<false>, 4),
    FP8NT_ENTRY("m_grouped_gemm_nn_ragged", ragged_rows<true>, 4),
    FP8NT_ENTRY("k_grouped_gemm_tn_ragged", ragged_weights, 5),
    FP8NT_ENTRY("group_rows_by_index", group_rows, 7),
    FP8NT_ENTRY("m_grouped_lora_add", lora_add, 8),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__torch_calls(void) { return PyModule_Create(&kModule); }
