// qmixer_usual.cpp -- the usual call of each mixer operator, checked and launched
// from C++: module _qmixer_usual, used by qmixer.py.
//
// A single token's kernels take 2 to 20 us; the same checks in Python take 10 more.
// Each function here answers a call whose operands are all as the operator
// wants them on the current device and stream, with an output of its own, and
// returns None for any other, without having launched anything: qmixer.py then
// goes its own way, which takes the rarer forms (outputs and streams of the
// caller's, other devices) and refuses the rest with a message.  Refusals of the
// C entry come before its first launch and are left to Python too; what it reports
// behind that, or what fails once it has returned, is raised: the state or residual
// may have moved on, so the call must not be made again.
#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "qmixer.h"

namespace {

using at::Tensor;

// Whether two tensors' memory is apart, by their bounds.
bool apart(const Tensor& a, const Tensor& b) {
    auto span = [](const Tensor& t) {
        int64_t n = 1;
        for (int d = 0; d < t.dim(); d++) n += (t.size(d) - 1) * t.stride(d);
        return n * (int64_t)t.element_size();
    };
    const char *pa = static_cast<const char*>(a.data_ptr()), *pb = static_cast<const char*>(b.data_ptr());
    return pa >= pb + span(b) || pb >= pa + span(a);
}

struct Call {
    bool ok = true;
    int device = -1;
    const Tensor* seen[16];          // the operands so far
    int n_seen = 0;

    // a CUDA tensor of the current device that no gradient is wanted for and that
    // carries no forward-mode tangent
    const Tensor* tensor(PyObject* o) {
        if (!ok || !THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        const Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.layout() != at::kStrided || t.is_neg() || t.is_conj()) ok = false;
        else if (device < 0) {
            device = t.get_device();
            if (device != c10::cuda::current_device()) ok = false;
        } else if (t.get_device() != device) ok = false;
        if (ok && t.requires_grad() && c10::GradMode::is_enabled()) ok = false;
        if (ok && t._fw_grad(0).defined()) ok = false;
        if (!ok) return nullptr;
        seen[n_seen++] = &t;
        return &t;
    }
    // whether the last operand, which the call writes, shares no memory with another
    bool last_alone() const {
        for (int i = 0; i + 1 < n_seen; i++)
            if (!apart(*seen[n_seen - 1], *seen[i])) return false;
        return true;
    }
    // nothing, or a contiguous vector of n
    const void* vector(PyObject* o, at::ScalarType type, int64_t n) {
        if (!ok || o == Py_None) return nullptr;
        const Tensor* t = tensor(o);
        if (!t || t->scalar_type() != type || t->dim() != 1 || t->size(0) != n || !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        return t->data_ptr();
    }
    void want(bool holds) { ok = ok && holds; }
    qstate_stream stream() const {
        return reinterpret_cast<qstate_stream>(c10::cuda::getCurrentCUDAStream(device).stream());
    }
};

int32_t code(const Tensor& t) {
    return t.scalar_type() == at::kFloat ? QSTATE_F32 : t.scalar_type() == at::kBFloat16 ? QSTATE_BF16 : -1;
}

// Stride between the rows of a tensor whose last `inner` dimensions are a row and whose
// leading ones walk in one stride; -1 for any other.
int64_t rows(const Tensor& t, int inner) {
    int64_t row = 1;
    const int n = (int)t.dim();
    for (int d = n - 1; d >= n - inner; d--) {
        if (t.size(d) != 1 && t.stride(d) != row) return -1;
        row *= t.size(d);
    }
    int64_t stride = -1, block = 1;          // tokens that one stride has covered
    for (int d = n - inner - 1; d >= 0; d--) {
        if (t.size(d) == 1) continue;
        if (stride < 0) stride = t.stride(d);
        else if (t.stride(d) != stride * block) return -1;
        block *= t.size(d);
    }
    if (stride < 0) return row;
    return stride < row ? -1 : stride;
}

// What a call has written in place, autograd learns by its version: an operation that
// saved the former values for its backward pass must not go on with these.
void written(const Tensor* t) {
    if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

bool on16(const Tensor& t) { return (reinterpret_cast<uintptr_t>(t.data_ptr()) & 15) == 0; }

PyObject* none() { Py_RETURN_NONE; }

// A call that may have launched.
struct Launched {
    const char* entry;
    int rc;
};

// Whether a C entry took its call; throws where it failed behind its checks.
bool taken(const char* entry, int rc) {
    if (rc == QSTATE_OK) return true;
    if (rc == QSTATE_EINVAL || rc == QSTATE_EUNSUPPORTED) return false;
    throw Launched{entry, rc};
}
// The outputs of a call that was taken, as Python objects (one, or a pair); `in_place`:
// what else it wrote, or NULL.
PyObject* wrapped(const char* entry, const Tensor* in_place, Tensor& y, Tensor* scales = nullptr) {
    try {
        written(in_place);
        PyObject* first = THPVariable_Wrap(std::move(y));
        if (!scales) return first;
        PyObject *second = THPVariable_Wrap(std::move(*scales)), *both = nullptr;
        if (first && second) both = PyTuple_Pack(2, first, second);
        Py_XDECREF(first);
        Py_XDECREF(second);
        return both;
    } catch (...) {
        throw Launched{entry, QSTATE_ENOMEM};
    }
}

// Sequences of a prompt with `lead` leading dimensions.
struct Prompt {
    int64_t sequences = 0, tokens = 0;
    const int32_t* starts = nullptr;
    Prompt(Call& c, const Tensor& x, int lead, PyObject* seq_starts) {
        if (lead == 2) {
            sequences = x.size(0);
            tokens = x.size(0) * x.size(1);
            c.want(seq_starts == Py_None);
            return;
        }
        sequences = 1;
        tokens = x.size(0);
        if (seq_starts == Py_None) return;
        const Tensor* s = c.tensor(seq_starts);
        if (!s || s->scalar_type() != at::kInt || s->dim() != 1 || s->size(0) < 2 || !s->is_contiguous()) {
            c.ok = false;
            return;
        }
        sequences = s->size(0) - 1;
        starts = static_cast<const int32_t*>(s->data_ptr());
    }
};

// ---------------------------------------------------------------- convolution
PyObject* conv_any(PyObject* const* a, bool step) {
    // x, weight, bias, state, activation [, initial, seq_starts]
    Call c;
    const Tensor* x = c.tensor(a[0]);
    if (!x || x->numel() == 0 || (step ? x->dim() != 2 : x->dim() != 2 && x->dim() != 3)) return none();
    const int32_t type = code(*x);
    const int64_t channels = x->size(-1), xs = rows(*x, 1);
    const Tensor* w = c.tensor(a[1]);
    if (!w || type < 0 || xs < 0 || w->scalar_type() != x->scalar_type() || w->dim() != 2 || w->size(0) != channels ||
        !w->is_contiguous() || channels > INT32_MAX)
        return none();
    const int64_t width = w->size(1);
    const void* bias = c.vector(a[2], x->scalar_type(), channels);
    Prompt p(c, *x, step ? 1 : (int)x->dim() - 1, step ? Py_None : a[6]);
    if (step) p.sequences = x->size(0);
    const Tensor* state = a[3] == Py_None ? nullptr : c.tensor(a[3]);
    const bool initial = !step && a[5] == Py_True;
    c.want(state || (!step && !initial));
    if (!c.ok || p.sequences > INT32_MAX || p.tokens > INT32_MAX) return none();
    if (state && (state->scalar_type() != x->scalar_type() || state->dim() != 3 || state->size(0) != p.sequences ||
                  state->size(1) != width - 1 || state->size(2) != channels || !state->is_contiguous() ||
                  !c.last_alone()))
        return none();
    Tensor y = at::empty(x->sizes(), x->options());
    const int32_t act = a[4] == Py_True ? QMIXER_SILU : 0;
    const char* const entry = step ? "qmixer_conv_step" : "qmixer_conv";
    int rc;
    if (step) {
        const qmixer_conv_step_args q{x->data_ptr(), xs, w->data_ptr(), bias, state->data_ptr(), y.data_ptr(), channels,
                                      (int32_t)x->size(0), (int32_t)channels, (int32_t)width, type, act};
        rc = qmixer_conv_step(&q, c.stream());
    } else {
        const qmixer_conv_args q{x->data_ptr(), xs, w->data_ptr(), bias, state ? state->data_ptr() : nullptr,
                                 y.data_ptr(), channels, p.starts, (int32_t)p.sequences, p.tokens, (int32_t)channels,
                                 (int32_t)width, type, act | (initial ? QMIXER_INITIAL : 0)};
        rc = qmixer_conv(&q, c.stream());
    }
    return taken(entry, rc) ? wrapped(entry, state, y) : none();
}

// ---------------------------------------------------------------- selective scan
PyObject* scan_any(PyObject* const* a, bool step) {
    // x, dt, A, B, C, D, dt_bias, state, softplus [, initial, seq_starts]
    Call c;
    const Tensor* x = c.tensor(a[0]);
    if (!x || x->numel() == 0 || (step ? x->dim() != 3 : x->dim() != 3 && x->dim() != 4)) return none();
    const int lead = (int)x->dim() - 2;
    const Tensor *dt = c.tensor(a[1]), *B = c.tensor(a[3]), *C = c.tensor(a[4]);
    if (!c.ok || B->dim() != x->dim() || dt->dim() != lead + 1 || B->sizes() != C->sizes()) return none();
    for (int d = 0; d < lead; d++) c.want(B->size(d) == x->size(d) && dt->size(d) == x->size(d));
    const int64_t heads = x->size(-2), d_v = x->size(-1), groups = B->size(-2), d_k = B->size(-1);
    const int32_t type = code(*x), dt_type = code(*dt);
    const int64_t xs = rows(*x, 2), dts = rows(*dt, 1), Bs = rows(*B, 2), Cs = rows(*C, 2), unit = 16 / x->element_size();
    c.want(type >= 0 && dt_type >= 0 && B->scalar_type() == x->scalar_type() && C->scalar_type() == x->scalar_type() &&
           dt->size(-1) == heads && groups > 0 && heads % groups == 0 && heads <= INT32_MAX && xs >= 0 && dts >= 0 &&
           Bs >= 0 && Cs >= 0 && xs % unit == 0 && Bs % unit == 0 && Cs % unit == 0 && on16(*x) && on16(*B) && on16(*C) &&
           a[2] != Py_None);
    const float* A = static_cast<const float*>(c.vector(a[2], at::kFloat, heads));
    const float* D = static_cast<const float*>(c.vector(a[5], at::kFloat, heads));
    const float* bias = static_cast<const float*>(c.vector(a[6], at::kFloat, heads));
    if (!c.ok) return none();
    Prompt p(c, *x, step ? 1 : lead, step ? Py_None : a[10]);
    if (step) p.sequences = x->size(0);
    const Tensor* state = a[7] == Py_None ? nullptr : c.tensor(a[7]);
    const bool initial = !step && a[9] == Py_True;
    c.want(state || (!step && !initial));
    if (!c.ok || p.sequences > INT32_MAX || p.tokens > INT32_MAX) return none();
    if (state && (state->scalar_type() != at::kFloat || state->dim() != 4 || state->size(0) != p.sequences ||
                  state->size(1) != heads || state->size(2) != d_k || state->size(3) != d_v || !state->is_contiguous() ||
                  !c.last_alone()))
        return none();
    const int32_t flags = (a[8] == Py_True ? QMIXER_SOFTPLUS : 0) | (initial ? QMIXER_INITIAL : 0);
    float* S = state ? static_cast<float*>(state->data_ptr()) : nullptr;
    if (step) {
        Tensor y = at::empty(x->sizes(), x->options());
        const qmixer_scan_step_args q{x->data_ptr(), xs, dt->data_ptr(), dts, A, B->data_ptr(), Bs, C->data_ptr(), Cs, D,
                                      bias, S, y.data_ptr(), heads * d_v, (int32_t)x->size(0), (int32_t)heads,
                                      (int32_t)groups, (int32_t)d_k, (int32_t)d_v, type, dt_type, flags};
        const char* const entry = "qmixer_scan_step";
        return taken(entry, qmixer_scan_step(&q, c.stream())) ? wrapped(entry, state, y) : none();
    }
    const int64_t bytes = qmixer_scan_workspace((int32_t)p.sequences, p.tokens, (int32_t)heads, (int32_t)groups,
                                                (int32_t)d_k, (int32_t)d_v, type);
    if (bytes < 0) return none();
    Tensor y = at::empty(x->sizes(), x->options()), work;
    if (bytes) work = at::empty({bytes}, x->options().dtype(at::kByte));
    const qmixer_scan_args q{x->data_ptr(), xs, dt->data_ptr(), dts, A, B->data_ptr(), Bs, C->data_ptr(), Cs, D, bias, S,
                             y.data_ptr(), heads * d_v, p.starts, (int32_t)p.sequences, p.tokens, (int32_t)heads,
                             (int32_t)groups, (int32_t)d_k, (int32_t)d_v, type, dt_type, flags,
                             bytes ? work.data_ptr() : nullptr, bytes};
    const char* const entry = "qmixer_scan";
    return taken(entry, qmixer_scan(&q, c.stream())) ? wrapped(entry, state, y) : none();
}

// ---------------------------------------------------------------- norm
PyObject* norm_any(PyObject* const* a) {
    // x, weight, other, before, eps, kind, group
    Call c;
    const Tensor* x = c.tensor(a[0]);
    if (!x || x->numel() == 0 || x->dim() < 1) return none();
    const int32_t type = code(*x);
    const int64_t columns = x->size(-1), xs = rows(*x, 1);
    const void* w = a[1] == Py_None ? nullptr : c.vector(a[1], x->scalar_type(), columns);
    const long before = PyLong_AsLong(a[3]), kind = PyLong_AsLong(a[5]), group = PyLong_AsLong(a[6]);
    const double eps = PyFloat_AsDouble(a[4]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return none();
    }
    c.want(type >= 0 && xs >= 0 && w && columns <= INT32_MAX && group >= 0 && (!group || (kind && columns % group == 0)));
    if (!c.ok) return none();
    const Tensor* other = nullptr;
    int64_t os = 0;
    if (before) {
        other = c.tensor(a[2]);
        if (!other || other->scalar_type() != x->scalar_type() || other->sizes() != x->sizes()) return none();
        os = rows(*other, 1);
        if (os < 0 || (before == QMIXER_BEFORE_RESIDUAL && !c.last_alone())) return none();
    }
    Tensor y = at::empty(x->sizes(), kind == QMIXER_OUT_INT8   ? x->options().dtype(at::kChar)
                                     : kind == QMIXER_OUT_E4M3 ? x->options().dtype(at::kFloat8_e4m3fn)
                                                               : x->options());
    Tensor scales;
    if (kind) {
        auto shape = x->sizes().vec();
        shape.back() = group ? columns / group : 1;
        scales = at::empty(shape, x->options().dtype(at::kFloat));
    }
    const qmixer_norm_args q{x->data_ptr(), xs, other ? other->data_ptr() : nullptr, os, w, y.data_ptr(), columns,
                             kind ? static_cast<float*>(scales.data_ptr()) : nullptr, x->numel() / columns,
                             (int32_t)columns, (int32_t)group, (float)eps, type, (int32_t)before, (int32_t)kind};
    const char* const entry = "qmixer_norm";
    if (!taken(entry, qmixer_norm(&q, c.stream()))) return none();
    return wrapped(entry, before == QMIXER_BEFORE_RESIDUAL ? other : nullptr, y, kind ? &scales : nullptr);
}

// ---------------------------------------------------------------- module
// No C++ exception leaves.  One in front of the launch, of a failed allocation, say,
// is left to the Python way, which meets it again and raises it.
template <class F> PyObject* guarded(F f) {
    try {
        return f();
    } catch (const Launched& e) {
        // QStateError(entry, code), as from Python
        PyErr_Clear();
        PyObject* const home = PyImport_ImportModule("bit_recurrent_state_decode_b200.qstate");
        PyObject* const type = home ? PyObject_GetAttrString(home, "QStateError") : nullptr;
        PyObject* const args = type ? Py_BuildValue("(si)", e.entry, e.rc) : nullptr;
        if (args) PyErr_SetObject(type, args);
        Py_XDECREF(args);
        Py_XDECREF(type);
        Py_XDECREF(home);
        return nullptr;
    } catch (...) {
        return none();
    }
}

PyObject* conv(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return n == 7 ? guarded([&] { return conv_any(a, false); }) : none();
}
PyObject* conv_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return n == 5 ? guarded([&] { return conv_any(a, true); }) : none();
}
PyObject* scan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return n == 11 ? guarded([&] { return scan_any(a, false); }) : none();
}
PyObject* scan_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return n == 9 ? guarded([&] { return scan_any(a, true); }) : none();
}
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return n == 7 ? guarded([&] { return norm_any(a); }) : none();
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(conv), ENTRY(conv_step), ENTRY(scan), ENTRY(scan_step), ENTRY(norm),
                         {nullptr, nullptr, 0, nullptr}};
// The versions of Python and PyTorch whose binary interface this is; build.py looks for it.
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmixer_usual", BUILT_FOR, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qmixer_usual(void) { return PyModule_Create(&module); }
