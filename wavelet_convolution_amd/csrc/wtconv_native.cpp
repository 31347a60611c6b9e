// The Python side of the expert rows and of the optimizer's step (argument
// marshalling only): tensors and lists of tensors to the plain pointers of the
// C-ABI, with the checks that those cannot carry. A list of hundreds of
// parameters is walked here because an attribute of a tensor costs Python 50
// to 100 ns: 330 gradients were 150 us that way, ten times the norm's own time.
//
// Every function takes positional arguments and enqueues on the current stream
// of the tensors' device, which has to be the current one: where it is not, the
// answer is NotImplemented, and the caller comes back from there. What a caller
// got wrong is a ValueError, what the library refuses is its status' WTConvError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <stdexcept>
#include <vector>

#include "../../include/wtconv.h"

namespace {

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct Raised {};      // Python's error is set
struct Elsewhere {};   // another device is the current one

template <class... A>
[[noreturn]] void refuse(const A&... parts) {
    std::ostringstream s;
    (s << ... << parts);
    throw Refused(s.str());
}

// Runs a function; its exceptions become Python's.
template <class F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const Raised&) {
    } catch (const Elsewhere&) {
        Py_RETURN_NOTIMPLEMENTED;
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        // torch's class of its own name, which its libraries do not export
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

void check_status(int status) {
    if (status == WTCONV_OK) return;
    PyObject* binding = PyImport_ImportModule("wavelet_convolution_amd.binding");
    if (binding) {
        PyObject* r = PyObject_CallMethod(binding, "_check", "i", status);
        Py_XDECREF(r);
        Py_DECREF(binding);
    }
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "libwtconv.so returned an error");
    throw Raised();
}

// A tensor argument on the device of the others.
const at::Tensor& tensor(const char* name, PyObject* o, const at::Tensor* like = nullptr) {
    if (!THPVariable_Check(o)) refuse(name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided) refuse(name, " must be a dense GPU tensor, got one on ", t.device());
    if (like && t.device() != like->device())
        refuse(name, " must be on ", like->device(), ", as the others; got one on ", t.device());
    return t;
}

void check_dense(const char* name, const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape) {
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
        refuse(name, " must be a contiguous ", type, " tensor of shape ", shape, "; got ", t.sizes(), " ",
               t.scalar_type(), t.is_contiguous() ? "" : ", not contiguous");
}
void check_buffer(const char* name, const at::Tensor& t, at::ScalarType type, int64_t n) {
    if (t.scalar_type() != type || t.numel() != n || !t.is_contiguous())
        refuse(name, " must be a contiguous ", type, " tensor of ", n, " elements; got ", t.sizes(), " ",
               t.scalar_type());
}
// One number on the GPU, or null.
const void* scalar(const char* name, PyObject* o, at::ScalarType type, const at::Tensor& like) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(name, o, &like);
    if (t.scalar_type() != type || t.numel() != 1)
        refuse(name, " must be a tensor of one ", type, " number; got ", t.sizes(), " ", t.scalar_type());
    return t.const_data_ptr();
}

int32_t dtype_code(at::ScalarType t) {
    return t == at::kFloat ? WTCONV_F32 : t == at::kBFloat16 ? WTCONV_BF16 : -1;
}

int64_t whole(const char* name, PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        if (!PyErr_ExceptionMatches(PyExc_OverflowError)) throw Raised();
        PyErr_Clear();
        refuse(name, " is out of range");
    }
    return v;
}
int32_t small(const char* name, int64_t v) {
    if (v < -(1ll << 31) || v >= 1ll << 31) refuse("sizes must be below 2^31; ", name, " is ", v);
    return (int32_t)v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1. && PyErr_Occurred()) throw Raised();
    return v;
}
// The current stream of the call's device, which is the current device.
void* stream_of(const at::Tensor& t) {
    if (t.get_device() != c10::hip::current_device()) throw Elsewhere();
    return (void*)c10::hip::getCurrentHIPStream(t.get_device()).stream();
}

// New memory on a tensor's device: what torch.empty does behind its dispatch.
at::Tensor fresh(const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type) {
    return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

// A workspace: the caller's, from its next multiple of 256 bytes on, or a new one.
struct Workspace {
    at::Tensor held;
    void* p = nullptr;
    size_t bytes = 0;
    Workspace(PyObject* given, size_t need, const at::Tensor& like) {
        if (given != Py_None) {
            held = tensor("ws", given, &like);
            if (!held.is_contiguous()) refuse("ws must be contiguous: its bytes are counted from its elements");
        } else if (need) {
            held = fresh(like, {(int64_t)need + 256}, at::kByte);
        } else {
            return;
        }
        const uintptr_t first = (uintptr_t)held.mutable_data_ptr(), at = (first + 255) & ~(uintptr_t)255;
        const size_t all = held.nbytes();
        p = (void*)at;
        bytes = all > at - first ? all - (at - first) : 0;
    }
};

// An output to write: the one given, checked, or a new one.
at::Tensor output(const char* name, PyObject* given, const at::Tensor& like, at::ScalarType type,
                  at::IntArrayRef shape) {
    if (given == Py_None) return fresh(like, shape, type);
    const at::Tensor& t = tensor(name, given, &like);
    check_dense(name, t, type, shape);
    return t;
}

// Autograd's own record of a change in place, as torch's operations keep it: a
// graph that needs what a tensor of the caller's held before raises an error.
void changed(PyObject* o) {
    if (o == Py_None) return;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// ------------------------------------------------------------- expert rows

PyObject* tuple_of(std::initializer_list<const at::Tensor*> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw Raised();
    Py_ssize_t i = 0;
    for (const at::Tensor* t : ts) {
        PyObject* o = t->defined() ? THPVariable_Wrap(*t) : (Py_INCREF(Py_None), Py_None);
        if (!o) {
            Py_DECREF(r);
            throw Raised();
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// expert, experts, order, place, offsets, ws
PyObject* expert_sort(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&] {
        const at::Tensor& e = tensor("expert", a[0]);
        void* const stream = stream_of(e);
        const bool wide = e.scalar_type() == at::kLong;
        if ((!wide && e.scalar_type() != at::kInt) || e.dim() < 2 || !e.is_contiguous())
            refuse("expert must be a contiguous int32 or int64 tensor [..., K]; got ", e.sizes(), " ", e.scalar_type(),
                   e.is_contiguous() ? "" : ", not contiguous");
        const int64_t k = e.size(-1), slots = e.numel(), experts = whole("experts", a[1]);
        if (k < 1) refuse("a row has at least one slot");
        const wtconv_expert_desc_t d{slots / k, small("K", k), small("experts", experts), 0, 0};
        const size_t need = wtconv_expert_workspace_size(&d);
        if (need == (size_t)-1)   // the call says what is wrong before it looks at a pointer
            check_status(wtconv_expert_sort(&d, nullptr, wide, nullptr, nullptr, nullptr, nullptr, 0, nullptr));
        const at::Tensor order = output("order", a[2], e, at::kInt, {slots});
        const at::Tensor place = output("place", a[3], e, at::kInt, e.sizes());
        const at::Tensor offsets = output("offsets", a[4], e, at::kInt, {experts + 1});
        const Workspace ws(a[5], need, e);
        check_status(wtconv_expert_sort(&d, e.const_data_ptr(), wide ? WTCONV_I64 : WTCONV_I32,
                                        order.mutable_data_ptr<int32_t>(), place.mutable_data_ptr<int32_t>(),
                                        offsets.mutable_data_ptr<int32_t>(), ws.p, ws.bytes, stream));
        for (int i : {2, 3, 4}) changed(a[i]);
        return tuple_of({&order, &place, &offsets});
    });
}

struct Route {
    const at::Tensor &place, &offsets;
    wtconv_expert_desc_t d;
    const int32_t *at, *ends;
};
Route route(PyObject* place_, PyObject* offsets_, const at::Tensor& rows) {
    const at::Tensor& place = tensor("place", place_, &rows);
    const at::Tensor& offsets = tensor("offsets", offsets_, &rows);
    if (place.scalar_type() != at::kInt || place.dim() < 2 || !place.is_contiguous())
        refuse("place must be a contiguous int32 tensor [..., K]; got ", place.sizes(), " ", place.scalar_type());
    if (offsets.scalar_type() != at::kInt || offsets.dim() != 1 || offsets.numel() < 2 || !offsets.is_contiguous())
        refuse("offsets must be a contiguous int32 tensor [E + 1]; got ", offsets.sizes(), " ", offsets.scalar_type());
    const int64_t k = place.size(-1), c = rows.dim() ? rows.size(-1) : 0;
    if (k < 1 || c < 1) refuse("a routing has at least one slot a row, and a row one channel; got K = ", k, ", C = ", c);
    return {place, offsets,
            {place.numel() / k, small("K", k), small("E", offsets.numel() - 1), small("C", c),
             dtype_code(rows.scalar_type())},
            place.const_data_ptr<int32_t>(), offsets.const_data_ptr<int32_t>()};
}
const at::Tensor& rows_arg(const char* name, PyObject* o) {
    const at::Tensor& t = tensor(name, o);
    if (dtype_code(t.scalar_type()) < 0 || t.dim() < 2 || !t.is_contiguous())
        refuse(name, " must be a contiguous float32 or bfloat16 tensor of rows [..., C]; got ", t.sizes(), " ",
               t.scalar_type(), t.is_contiguous() ? "" : ", not contiguous");
    return t;
}
void check_token_rows(const char* name, const at::Tensor& t, const at::Tensor& place) {
    if (t.sizes().slice(0, t.dim() - 1) != place.sizes().slice(0, place.dim() - 1))
        refuse(name, " must have place's rows, ", place.sizes().slice(0, place.dim() - 1), " and C; got ", t.sizes());
}
void check_sorted_rows(const char* name, const at::Tensor& t, const at::Tensor& place) {
    if (t.dim() != 2 || t.size(0) != place.numel())
        refuse(name, " must have one row a slot, [", place.numel(), ", C]; got ", t.sizes());
}
std::vector<int64_t> token_shape(const at::Tensor& place, int64_t c) {
    std::vector<int64_t> s(place.sizes().begin(), place.sizes().end());
    s.back() = c;
    return s;
}

// x, place, offsets, xs
PyObject* expert_rows_fwd(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&] {
        const at::Tensor& x = rows_arg("x", a[0]);
        void* const stream = stream_of(x);
        const Route r = route(a[1], a[2], x);
        check_token_rows("x", x, r.place);
        const at::Tensor xs = output("xs", a[3], x, x.scalar_type(), {r.place.numel(), x.size(-1)});
        check_status(wtconv_expert_rows_fwd(&r.d, x.const_data_ptr(), r.at, r.ends, xs.mutable_data_ptr(),
                                            stream));
        changed(a[3]);
        return THPVariable_Wrap(xs);
    });
}

// dxs, place, offsets, dx
PyObject* expert_rows_bwd(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&] {
        const at::Tensor& dxs = rows_arg("dxs", a[0]);
        void* const stream = stream_of(dxs);
        const Route r = route(a[1], a[2], dxs);
        check_sorted_rows("dxs", dxs, r.place);
        const at::Tensor dx = output("dx", a[3], dxs, dxs.scalar_type(), token_shape(r.place, dxs.size(-1)));
        check_status(wtconv_expert_rows_bwd(&r.d, dxs.const_data_ptr(), r.at, r.ends, dx.mutable_data_ptr(),
                                            stream));
        changed(a[3]);
        return THPVariable_Wrap(dx);
    });
}

// ys, weight, place, offsets, y
PyObject* expert_sum_fwd(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&] {
        const at::Tensor& ys = rows_arg("ys", a[0]);
        void* const stream = stream_of(ys);
        const Route r = route(a[2], a[3], ys);
        check_sorted_rows("ys", ys, r.place);
        const at::Tensor& w = tensor("weight", a[1], &ys);
        check_dense("weight", w, at::kFloat, r.place.sizes());
        const at::Tensor y = output("y", a[4], ys, ys.scalar_type(), token_shape(r.place, ys.size(-1)));
        check_status(wtconv_expert_sum_fwd(&r.d, ys.const_data_ptr(), w.const_data_ptr<float>(), r.at, r.ends,
                                           y.mutable_data_ptr(), stream));
        changed(a[4]);
        return THPVariable_Wrap(y);
    });
}

// dy, ys, weight, place, offsets, want dys, want dweight, dys, dweight
PyObject* expert_sum_bwd(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&] {
        const at::Tensor& dy = rows_arg("dy", a[0]);
        void* const stream = stream_of(dy);
        const Route r = route(a[3], a[4], dy);
        check_token_rows("dy", dy, r.place);
        const bool want_dys = a[5] == Py_True, want_dw = a[6] == Py_True;
        const void* ys_at = nullptr;
        const float* w_at = nullptr;
        if (want_dw || a[1] != Py_None) {
            const at::Tensor& ys = tensor("ys", a[1], &dy);
            check_dense("ys", ys, dy.scalar_type(), {r.place.numel(), dy.size(-1)});
            ys_at = ys.const_data_ptr();
        }
        if (want_dys || a[2] != Py_None) {
            const at::Tensor& w = tensor("weight", a[2], &dy);
            check_dense("weight", w, at::kFloat, r.place.sizes());
            w_at = w.const_data_ptr<float>();
        }
        at::Tensor dys, dw;
        if (want_dys) dys = output("dys", a[7], dy, dy.scalar_type(), {r.place.numel(), dy.size(-1)});
        if (want_dw) dw = output("dweight", a[8], dy, at::kFloat, r.place.sizes());
        check_status(wtconv_expert_sum_bwd(&r.d, dy.const_data_ptr(), ys_at, w_at, r.at, r.ends,
                                           dys.defined() ? dys.mutable_data_ptr() : nullptr,
                                           dw.defined() ? dw.mutable_data_ptr<float>() : nullptr, stream));
        if (want_dys) changed(a[7]);
        if (want_dw) changed(a[8]);
        return tuple_of({&dys, &dw});
    });
}

// ------------------------------------------------------- lists of tensors

// A sequence's items, held while it lives.
struct Items {
    PyObject* held;
    PyObject** o;
    int32_t n;
    Items(const char* name, PyObject* seq) : held(PySequence_Fast(seq, "a sequence is required")) {
        if (!held) throw Raised();
        const Py_ssize_t size = PySequence_Fast_GET_SIZE(held);
        if (size > 1 << 24) {
            Py_DECREF(held);
            refuse("too many ", name);
        }
        o = PySequence_Fast_ITEMS(held);
        n = (int32_t)size;
    }
    ~Items() { Py_DECREF(held); }
    Items(const Items&) = delete;
};

// A contiguous tensor of a list, on the device of the others.
const at::Tensor& listed(const char* name, PyObject* o, const at::Tensor*& like) {
    const at::Tensor& t = tensor(name, o, like);
    if (!like) like = &t;
    if (!t.is_contiguous()) refuse(name, " must be contiguous tensors; got one with strides ", t.strides());
    return t;
}

// n fp32 numbers on the host: one for all, a CPU tensor, or a sequence of them.
const float* each(const char* name, PyObject* o, int32_t n, std::vector<float>& own) {
    if (THPVariable_Check(o)) {
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cpu() || t.scalar_type() != at::kFloat || t.numel() != n || !t.is_contiguous())
            refuse(name, " must be a number, or one for each of the ", n, " tensors (a contiguous float32 tensor on the ",
                   "host, or a sequence); got ", t.sizes(), " ", t.scalar_type(), " on ", t.device());
        return t.const_data_ptr<float>();
    }
    if (PyFloat_Check(o) || PyLong_Check(o)) {
        own.assign(n, (float)real(o));
        return own.data();
    }
    const Items items(name, o);
    if (items.n != n) refuse(name, " must be a number, or one for each of the ", n, " tensors; got ", items.n);
    own.resize(n);
    for (int32_t i = 0; i < n; ++i) own[i] = (float)real(items.o[i]);
    return own.data();
}

// params (a list of tensors; their sizes count only)
PyObject* adamw_state_count(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&] {
        const Items params("params", a[0]);
        std::vector<int64_t> counts(params.n);
        for (int32_t i = 0; i < params.n; ++i) {
            if (!THPVariable_Check(params.o[i])) refuse("params must be tensors, got ", Py_TYPE(params.o[i])->tp_name);
            counts[i] = THPVariable_Unpack(params.o[i]).numel();
        }
        const int64_t n = wtconv_adamw_state_count(counts.data(), params.n);
        if (n < 0) check_status(WTCONV_ERR_UNSUPPORTED_SHAPE);
        return PyLong_FromLongLong(n);
    });
}

// The arguments of a step as the C-ABI takes them, from
// params, grads, m, v, step, lr, weight_decay, beta1, beta2, eps, scales, master, factor, lr_factor, rng, site
struct AdamwCall {
    const Items params, grads;
    const int32_t n;
    std::vector<void*> p;
    std::vector<const void*> g;
    std::vector<int64_t> counts;
    const at::Tensor* like = nullptr;
    void *m, *v;
    float *scales = nullptr, *master = nullptr;
    const int64_t* step;
    const float *factor, *lr_factor, *lr, *wd;
    const uint64_t* rng = nullptr;
    std::vector<float> own_lr, own_wd;
    wtconv_adamw_desc_t d;

    explicit AdamwCall(PyObject* const* a) : params("params", a[0]), grads("grads", a[1]), n(params.n) {
        if (n != grads.n || n == 0)
            refuse("one gradient (or None) a parameter, and one at least, are required; got ", n, " and ", grads.n);
        p.resize(n);
        g.resize(n);
        counts.resize(n);
        int32_t ptype = -1, gtype = -1;
        for (int32_t i = 0; i < n; ++i) {
            const at::Tensor& t = listed("params", params.o[i], like);
            const int32_t code = dtype_code(t.scalar_type());
            if (code < 0 || (ptype >= 0 && code != ptype))
                refuse("params must be all float32 or all bfloat16; got ", t.scalar_type());
            ptype = code;
            p[i] = t.mutable_data_ptr();
            counts[i] = t.numel();
            if (grads.o[i] == Py_None) continue;
            const at::Tensor& u = listed("grads", grads.o[i], like);
            const int32_t gcode = dtype_code(u.scalar_type());
            if (gcode < 0 || (gtype >= 0 && gcode != gtype))
                refuse("grads must be all float32 or all bfloat16; got ", u.scalar_type());
            gtype = gcode;
            if (u.sizes() != t.sizes())
                refuse("gradients must have their parameters' shapes; got ", u.sizes(), " for ", t.sizes());
            g[i] = u.const_data_ptr();
        }
        const int64_t all = wtconv_adamw_state_count(counts.data(), n);
        if (all < 0) check_status(WTCONV_ERR_UNSUPPORTED_SHAPE);
        const bool eight = a[10] != Py_None;
        const at::ScalarType kind = eight ? at::kFloat8_e4m3fn : at::kFloat;
        const at::Tensor &m_ = tensor("m", a[2], like), &v_ = tensor("v", a[3], like);
        check_buffer("m", m_, kind, all);
        check_buffer("v", v_, kind, all);
        m = m_.mutable_data_ptr();
        v = v_.mutable_data_ptr();
        if (eight) {
            const at::Tensor& t = tensor("scales", a[10], like);
            check_buffer("scales", t, at::kFloat, all / WTCONV_ADAMW_BLOCK * 2);
            scales = t.mutable_data_ptr<float>();
        }
        if (a[11] != Py_None) {
            const at::Tensor& t = tensor("master", a[11], like);
            if (ptype != WTCONV_BF16) refuse("master copies are for bfloat16 parameters");
            check_buffer("master", t, at::kFloat, all);
            master = t.mutable_data_ptr<float>();
        }
        if (a[4] == Py_None) refuse("step, one int64 number on the GPU, is required");
        step = (const int64_t*)scalar("step", a[4], at::kLong, *like);
        factor = (const float*)scalar("factor", a[12], at::kFloat, *like);
        lr_factor = (const float*)scalar("lr_factor", a[13], at::kFloat, *like);
        if (a[14] != Py_None) {
            const at::Tensor& t = tensor("rng", a[14], like);
            if (!eight || t.scalar_type() != at::kLong || t.numel() != 2 || !t.is_contiguous())
                refuse("rng must be a contiguous int64 tensor {seed, offset}, for states in 8 bits");
            rng = (const uint64_t*)t.const_data_ptr();
        }
        const int64_t site = whole("site", a[15]);
        if (site < 0 || site >= 1ll << 31) refuse("site must be in 0..2^31-1");
        lr = each("lr", a[5], n, own_lr);
        wd = each("weight_decay", a[6], n, own_wd);
        d = {ptype, gtype < 0 ? WTCONV_F32 : gtype, eight ? 8 : 32, (int32_t)site, real(a[7]), real(a[8]), real(a[9])};
    }
};

PyObject* adamw_check(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const AdamwCall c(a);
        check_status(wtconv_adamw_check(&c.d, c.n, c.p.data(), c.g.data(), c.counts.data(), c.lr, c.wd, c.m, c.v,
                                        c.scales, c.master, c.step, c.factor, c.lr_factor, c.rng));
        Py_RETURN_NONE;
    });
}

PyObject* adamw_step(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const AdamwCall c(a);
        void* const stream = stream_of(*c.like);
        check_status(wtconv_adamw_step(&c.d, c.n, c.p.data(), c.g.data(), c.counts.data(), c.lr, c.wd, c.m, c.v,
                                       c.scales, c.master, c.step, c.factor, c.lr_factor, c.rng, stream));
        bool any = false;
        for (int32_t i = 0; i < c.n; ++i)
            if (c.g[i]) {
                changed(c.params.o[i]);
                any = true;
            }
        if (any)
            for (int i : {2, 3, 10, 11}) changed(a[i]);
        Py_RETURN_NONE;
    });
}

// grads, max_norm, step, out, ws
PyObject* grad_norm(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&] {
        const Items grads("grads", a[0]);
        std::vector<const void*> g(grads.n);
        std::vector<int64_t> counts(grads.n);
        std::vector<int32_t> types(grads.n);
        const at::Tensor* like = nullptr;
        int32_t n = 0;
        for (int32_t i = 0; i < grads.n; ++i) {
            if (grads.o[i] == Py_None) continue;
            const at::Tensor& t = listed("grads", grads.o[i], like);
            types[n] = dtype_code(t.scalar_type());
            if (types[n] < 0) refuse("gradients must be float32 or bfloat16; got ", t.scalar_type());
            counts[n] = t.numel();
            g[n++] = t.const_data_ptr();
        }
        if (n == 0) refuse("at least one gradient is required");
        void* const stream = stream_of(*like);
        const double most = real(a[1]);
        if (!(most > 0)) refuse("max_norm must be above 0 (infinity: no clipping); got ", most);
        const at::Tensor out = output("out", a[3], *like, at::kFloat, {2});
        const void* step = scalar("step", a[2], at::kLong, *like);
        const size_t need = wtconv_grad_norm_workspace_size(counts.data(), n);
        if (need == (size_t)-1) check_status(WTCONV_ERR_UNSUPPORTED_SHAPE);
        const Workspace ws(a[4], need, *like);
        check_status(wtconv_grad_norm(n, g.data(), counts.data(), types.data(), most, (int64_t*)step,
                                      out.mutable_data_ptr<float>(), ws.p, ws.bytes, stream));
        changed(a[2]);
        changed(a[3]);
        return THPVariable_Wrap(out);
    });
}

// The number of arguments is the caller's in this package; a wrong one would
// read past the array.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), int N>
PyObject* counted(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments are required, got %zd", N, n);
        return nullptr;
    }
    return F(self, a, n);
}
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), int N>
PyMethodDef method(const char* name) {
    return {name, (PyCFunction)(void (*)(void)) & counted<F, N>, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<expert_sort, 6>("expert_sort"),
    method<expert_rows_fwd, 4>("expert_rows_fwd"),
    method<expert_rows_bwd, 4>("expert_rows_bwd"),
    method<expert_sum_fwd, 5>("expert_sum_fwd"),
    method<expert_sum_bwd, 9>("expert_sum_bwd"),
    method<adamw_state_count, 1>("adamw_state_count"),
    method<adamw_check, 16>("adamw_check"),
    method<adamw_step, 16>("adamw_step"),
    method<grad_norm, 5>("grad_norm"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
