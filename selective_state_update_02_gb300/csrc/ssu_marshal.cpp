// Marshalling of the prompt, rotation and attention calls from Python: one look at every tensor,
// the ABI's structs, and the C entry points by the addresses that bind() was given.
//
// These calls sit in a serving loop beside the decode step and are often shorter on the device than
// their marshalling: attribute by attribute from Python it took 7.3 us of a rotation's call (a
// tensor's sizes, strides, type, device and address some 80 ns each); here it takes 0.7, and a
// call of 8 tokens 3.0 instead of 10.6.
// A refusal raises TypeError or ValueError; a call's ssu_status_t is returned.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <exception>
#include <initializer_list>
#include <string>

#include "ssu.h"

namespace {

using at::Tensor;

decltype(&ssu_update_prompts) update_prompts_fn;
decltype(&ssu_rotate_qk) rotate_qk_fn;
decltype(&ssu_attend) attend_fn;

struct Refusal {
    PyObject *type;
    std::string text;
};

[[noreturn]] void refuse_type(const std::string &text) { throw Refusal{PyExc_TypeError, text}; }
[[noreturn]] void refuse(const std::string &text) { throw Refusal{PyExc_ValueError, text}; }

std::string listed(at::IntArrayRef sizes) {
    std::string s = "[";
    for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
    return s + "]";
}

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

// The tensor at `o`, of one of two types (the same one twice where there is no choice) and numbers
// of dimensions.
const Tensor &operand(PyObject *o, const char *name, at::ScalarType type, at::ScalarType other,
                      int dims, int other_dims) {
    const Tensor &t = tensor(o, name);
    const at::ScalarType got = t.scalar_type();
    if ((got != type && got != other) || (t.dim() != dims && t.dim() != other_dims))
        refuse_type(std::string(name) + " must be " + toString(type) +
                    (type == other ? std::string() : std::string(" or ") + toString(other)) +
                    " with " + std::to_string(dims) +
                    (dims == other_dims ? std::string() : " or " + std::to_string(other_dims)) +
                    " dims, got " + toString(got) + " with " + std::to_string(t.dim()));
    return t;
}

const Tensor &bf16(PyObject *o, const char *name, int dims) {
    return operand(o, name, at::kBFloat16, at::kBFloat16, dims, dims);
}

const Tensor &fp32(PyObject *o, const char *name, int dims, int other_dims) {
    return operand(o, name, at::kFloat, at::kFloat, dims, other_dims);
}

const Tensor &index(PyObject *o, const char *name, int dims) {
    return operand(o, name, at::kInt, at::kLong, dims, dims);
}

const Tensor &index_like(PyObject *o, const char *name, int dims, const Tensor &like) {
    return operand(o, name, like.scalar_type(), like.scalar_type(), dims, dims);
}

int32_t index_dtype(const Tensor &t) {
    return t.scalar_type() == at::kLong ? SSU_INDEX_I64 : SSU_INDEX_I32;
}

void shaped(const Tensor &t, const char *name, std::initializer_list<int64_t> want) {
    if (t.sizes() != at::IntArrayRef(want))
        refuse(std::string(name) + " must have the shape " + listed(want) + ", got " +
               listed(t.sizes()));
}

// The CUDA device of every operand.
int device_of(std::initializer_list<const Tensor *> operands) {
    const int device = static_cast<int>((*operands.begin())->get_device());
    for (const Tensor *t : operands)
        if (!t->is_cuda() || t->get_device() != device)
            refuse("every operand must be a CUDA tensor of one device, got " +
                   (*operands.begin())->device().str() + " and " + t->device().str());
    return device;
}

template <typename T = void>
T *at_device(const Tensor &t) {
    return static_cast<T *>(t.data_ptr());
}

uint16_t *bits(const Tensor &t) { return at_device<uint16_t>(t); }

// Strides of the leading dimensions; those that the tensor does not have are broadcast.
void strides_of(const Tensor &t, int dims, int64_t *to) {
    for (int i = 0; i < dims; ++i) to[i] = i < t.dim() ? t.stride(i) : 0;
}

// The same of a per-head operand in its expanded form.
void head_strides(const Tensor &t, const char *name, std::initializer_list<int64_t> full,
                  int64_t *to) {
    if (t.sizes() != at::IntArrayRef(full).slice(0, t.dim()))
        refuse(std::string(name) + " must have the shape " + listed(full) + " or " +
               listed(at::IntArrayRef(full).slice(0, 1)) + ", got " + listed(t.sizes()));
    strides_of(t, static_cast<int>(full.size()), to);
}

struct Workspace {
    void *at = nullptr;
    int64_t bytes = 0;
};

Workspace workspace(PyObject *o, int device) {
    Workspace w;
    if (o == Py_None) return w;
    const Tensor &t = tensor(o, "workspace");
    if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous())
        refuse("workspace must be a contiguous CUDA tensor of the operands' device");
    w.at = t.data_ptr();
    w.bytes = static_cast<int64_t>(t.nbytes());
    return w;
}

// A failed conversion leaves Python's error set; `call` looks for it before the entry point runs.
void *pointer(PyObject *o) { return o == Py_None ? nullptr : PyLong_AsVoidPtr(o); }

struct Failed {};

template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F body) {
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, got);
        return nullptr;
    }
    try {
        return PyLong_FromLong(body());
    } catch (const Refusal &r) {
        PyErr_SetString(r.type, r.text.c_str());
    } catch (const Failed &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// The C call, without the interpreter's lock.  Its arguments are worked out before, with the lock
// held: asking a tensor without storage for its address throws.
template <typename F, typename... Args>
long call(F entry, Args... args) {
    struct Unlocked {
        PyThreadState *const thread = PyEval_SaveThread();
        ~Unlocked() { PyEval_RestoreThread(thread); }
    };
    if (PyErr_Occurred()) throw Failed{};
    const Unlocked unlocked;
    return entry(args...);
}

// handle, state_pool, state_batch_indices, cu_tokens, x, dt, dt_bias, A, B, C, D, out, workspace,
// fresh, stream
PyObject *update_prompts(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        const Tensor &pool = operand(a[1], "state_pool", at::kFloat, at::kBFloat16, 4, 4);
        const Tensor &cu = index(a[3], "cu_tokens", 1);
        const Tensor &slots = index_like(a[2], "state_batch_indices", 1, cu);
        const Tensor &x = bf16(a[4], "x", 3);
        const Tensor &dt = operand(a[5], "dt", at::kBFloat16, at::kBFloat16, 2, 3);
        const Tensor &dt_bias = fp32(a[6], "dt_bias", 1, 2), &A = fp32(a[7], "A", 1, 3);
        const Tensor &B = bf16(a[8], "B", 3), &C = bf16(a[9], "C", 3);
        const Tensor &D = fp32(a[10], "D", 1, 2), &out = bf16(a[11], "out", 3);
        const int64_t H = pool.size(1), P = pool.size(2), N = pool.size(3);
        const int64_t T = B.size(0), G = B.size(1), bs = slots.size(0);
        shaped(x, "x", {T, H, P});
        shaped(out, "out", {T, H, P});
        shaped(B, "B", {T, G, N});
        shaped(C, "C", {T, G, N});
        if (dt.dim() == 2)
            shaped(dt, "dt", {T, H});
        else
            shaped(dt, "dt", {T, H, P});
        if (cu.size(0) != bs + 1 || !cu.is_contiguous())
            refuse("cu_tokens must be contiguous with " + std::to_string(bs + 1) + " entries");
        const int device = device_of(
            {&pool, &slots, &cu, &x, &dt, &dt_bias, &A, &B, &C, &D, &out});
        const uint8_t *fresh = nullptr;
        if (a[13] != Py_None) {
            const Tensor &f = tensor(a[13], "fresh");
            if ((f.scalar_type() != at::kByte && f.scalar_type() != at::kBool) ||
                f.sizes() != slots.sizes() || !f.is_contiguous() || !f.is_cuda() ||
                f.get_device() != device)
                refuse("fresh must be a contiguous uint8 or bool CUDA tensor with one entry per "
                       "prompt");
            fresh = at_device<uint8_t>(f);
        }
        const ssu_shape_t shape = {bs, H, P, N, G, pool.size(0), index_dtype(cu),
                                   pool.scalar_type() == at::kFloat ? SSU_STATE_F32
                                                                    : SSU_STATE_BF16};
        ssu_strides_t st;
        strides_of(pool, 4, st.state);
        strides_of(x, 3, st.x);
        strides_of(out, 3, st.out);
        strides_of(dt, 3, st.dt);
        strides_of(B, 3, st.B);
        strides_of(C, 3, st.C);
        head_strides(dt_bias, "dt_bias", {H, P}, st.dt_bias);
        head_strides(D, "D", {H, P}, st.D);
        head_strides(A, "A", {H, P, N}, st.A);
        st.idx = slots.stride(0);
        const Workspace w = workspace(a[12], device);
        auto *handle = static_cast<ssu_handle_t>(pointer(a[0]));
        auto *stream = static_cast<ssu_stream_t>(pointer(a[14]));
        return call(update_prompts_fn, handle, at_device(pool), at_device(slots), at_device(cu),
                    fresh, bits(x), bits(dt), at_device<float>(dt_bias), at_device<float>(A),
                    bits(B), bits(C), at_device<float>(D), bits(out), &shape, &st, T, w.at, w.bytes,
                    stream);
    });
}

// handle, q, k, v, q_weight, k_weight, table, positions, q_out, k_pages, v_pages, slots, eps,
// interleaved, stream
PyObject *rotate_qk(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        const Tensor &q = bf16(a[1], "q", 3), &k = bf16(a[2], "k", 3), &v = bf16(a[3], "v", 3);
        const Tensor &q_weight = fp32(a[4], "q_weight", 1, 1);
        const Tensor &k_weight = fp32(a[5], "k_weight", 1, 1), &table = fp32(a[6], "table", 2, 2);
        const Tensor &slots = index(a[11], "slots", 1);
        const Tensor &positions = index_like(a[7], "positions", 1, slots);
        const Tensor &q_out = bf16(a[8], "q_out", 3);
        const Tensor &k_pages = bf16(a[9], "k_pages", 4), &v_pages = bf16(a[10], "v_pages", 4);
        const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hk = k.size(1);
        shaped(q_out, "q_out", {T, Hq, D});
        shaped(k, "k", {T, Hk, D});
        shaped(v, "v", {T, Hk, D});
        const int64_t pages = k_pages.size(0), page = k_pages.size(1);
        shaped(k_pages, "k_pages", {pages, page, Hk, D});
        shaped(v_pages, "v_pages", {pages, page, Hk, D});
        shaped(q_weight, "q_weight", {D});
        shaped(k_weight, "k_weight", {D});
        shaped(positions, "positions", {T});
        shaped(slots, "slots", {T});
        if (q.stride(2) != 1 || k.stride(2) != 1 || v.stride(2) != 1 || q_out.stride(2) != 1 ||
            k_pages.stride(3) != 1 || v_pages.stride(3) != 1 || table.stride(1) != 1 ||
            q_weight.stride(0) != 1 || k_weight.stride(0) != 1)
            refuse("the last dimension of every operand must have stride 1");
        device_of({&q, &k, &v, &q_weight, &k_weight, &table, &positions, &q_out, &k_pages,
                   &v_pages, &slots});
        const int interleaved = PyObject_IsTrue(a[13]);
        const ssu_rotate_shape_t shape = {T,     Hq,   Hk,
                                          D,     table.size(1), table.size(0),
                                          pages, page, index_dtype(slots),
                                          interleaved};
        ssu_rotate_strides_t st;
        strides_of(q, 2, st.q);
        strides_of(k, 2, st.k);
        strides_of(v, 2, st.v);
        strides_of(q_out, 2, st.q_out);
        strides_of(k_pages, 3, st.k_pages);
        strides_of(v_pages, 3, st.v_pages);
        st.table = table.stride(0);
        st.positions = positions.stride(0);
        st.slots = slots.stride(0);
        const float eps = static_cast<float>(PyFloat_AsDouble(a[12]));
        auto *handle = static_cast<ssu_handle_t>(pointer(a[0]));
        auto *stream = static_cast<ssu_stream_t>(pointer(a[14]));
        return call(rotate_qk_fn, handle, bits(q), bits(k), bits(v), at_device<float>(q_weight),
                    at_device<float>(k_weight), at_device<float>(table), at_device(positions),
                    bits(q_out), bits(k_pages), bits(v_pages), at_device(slots), &shape, &st, eps,
                    stream);
    });
}

// handle, q, k_pages, v_pages, page_table, lengths, out, workspace, scale, window, sinks, stream
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        const Tensor &q = bf16(a[1], "q", 3), &out = bf16(a[6], "out", 3);
        const Tensor &k_pages = bf16(a[2], "k_pages", 4), &v_pages = bf16(a[3], "v_pages", 4);
        const Tensor &lengths = index(a[5], "lengths", 1);
        const Tensor &page_table = index_like(a[4], "page_table", 2, lengths);
        const int64_t bs = q.size(0), Hq = q.size(1), D = q.size(2);
        const int64_t pages = k_pages.size(0), page = k_pages.size(1), Hk = k_pages.size(2);
        shaped(out, "out", {bs, Hq, D});
        shaped(k_pages, "k_pages", {pages, page, Hk, D});
        shaped(v_pages, "v_pages", {pages, page, Hk, D});
        shaped(page_table, "page_table", {bs, page_table.size(1)});
        shaped(lengths, "lengths", {bs});
        if (q.stride(2) != 1 || out.stride(2) != 1 || k_pages.stride(3) != 1 ||
            v_pages.stride(3) != 1)
            refuse("the last dimension of q, out and the pages must have stride 1");
        const int device = device_of({&q, &k_pages, &v_pages, &page_table, &lengths, &out});
        const Workspace w = workspace(a[7], device);
        const ssu_attend_shape_t shape = {bs,   Hq, Hk, D, pages, page, page_table.size(1),
                                          index_dtype(lengths), 0};
        ssu_attend_strides_t st;
        strides_of(q, 2, st.q);
        strides_of(out, 2, st.out);
        strides_of(k_pages, 3, st.k_pages);
        strides_of(v_pages, 3, st.v_pages);
        strides_of(page_table, 2, st.page_table);
        st.lengths = lengths.stride(0);
        const double scale =
            a[8] == Py_None ? 1.0 / std::sqrt(static_cast<double>(D)) : PyFloat_AsDouble(a[8]);
        const int64_t window = PyLong_AsLongLong(a[9]), sinks = PyLong_AsLongLong(a[10]);
        auto *handle = static_cast<ssu_handle_t>(pointer(a[0]));
        auto *stream = static_cast<ssu_stream_t>(pointer(a[11]));
        return call(attend_fn, handle, bits(q), bits(k_pages), bits(v_pages), at_device(page_table),
                    at_device(lengths), bits(out), &shape, &st, static_cast<float>(scale), window,
                    sinks, w.at, w.bytes, stream);
    });
}

// Addresses of ssu_update_prompts, ssu_rotate_qk and ssu_attend.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 3, [&] {
        update_prompts_fn = reinterpret_cast<decltype(update_prompts_fn)>(pointer(a[0]));
        rotate_qk_fn = reinterpret_cast<decltype(rotate_qk_fn)>(pointer(a[1]));
        attend_fn = reinterpret_cast<decltype(attend_fn)>(pointer(a[2]));
        if (PyErr_Occurred()) throw Failed{};
        return 0L;
    });
}

template <PyObject *(*kFunction)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kFunction)),
            METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<update_prompts>("update_prompts"), method<rotate_qk>("rotate_qk"),
                         method<attend>("attend"), method<bind>("bind"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                          nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module_def); }
