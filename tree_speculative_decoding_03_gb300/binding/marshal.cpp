// marshal.cpp -- argument marshalling of the serving operators: torch tensors to the C ABI.
//
// A decoding step calls these three operators once per layer or step, each on up to fifteen
// tensors whose types, shapes and devices have to be checked; in Python that costs more than the
// launch (13 - 16 us a call on a Grace core, of which 5 - 8 us the launches).  Each function takes
// the address of the library's entry point, the tensors and the raw stream (None: torch's current
// one), checks, calls, and returns the entry's status.
#include <Python.h>

#include <stdexcept>
#include <string>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tsv.h"

namespace {

// What a caller got wrong; raised as ValueError.
struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

std::string text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a torch tensor");
    return THPVariable_Unpack(o);
}

const at::Tensor& ranked(PyObject* o, const char* name, int dim) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != dim) throw Refused(std::string(name) + " must have " + std::to_string(dim) + " dimensions, not " + text(t.sizes()));
    return t;
}

void* need(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) {
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
        throw Refused(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor of shape " + text(shape) +
                      ", not " + c10::toString(t.scalar_type()) + " " + text(t.sizes()));
    return t.data_ptr();
}

int small(int64_t x, const char* name) {
    if (x < 0 || x > 0x7fffffff) throw Refused(std::string(name) + " does not fit 32 bits");
    return static_cast<int>(x);
}

tsv_dtype dtype_of(const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return TSV_BF16;
    if (t.scalar_type() == at::kFloat) return TSV_F32;
    throw Refused(std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
}

// All tensors on the current device; the stream to launch on.
void* stream_for(PyObject* stream, std::initializer_list<const at::Tensor*> ts) {
    int dev = -1;
    for (const at::Tensor* t : ts) {
        if (t == nullptr) continue;
        if (!t->is_cuda()) throw Refused("tensors must be on a CUDA device");
        if (dev < 0) dev = t->get_device();
        if (t->get_device() != dev) throw Refused("tensors must be on one CUDA device");
    }
    if (c10::cuda::current_device() != dev) throw Refused("tensors must be on the current CUDA device");
    if (stream == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    return PyLong_AsVoidPtr(stream);
}

template <typename F>
F entry(PyObject* address) {
    return reinterpret_cast<F>(PyLong_AsVoidPtr(address));
}

// Runs a body that returns a tsv_status; C++ exceptions become Python ones.
template <typename Body>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, Body body) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        const int st = body();
        return PyErr_Occurred() ? nullptr : PyLong_FromLong(st);
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

template <typename F, typename... A>
int call(F f, A... args) {
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = f(args...);
    Py_END_ALLOW_THREADS
    return st;
}

// (entry, seq_lens, new_lens, block_table, blocks_held, blocks_held_out, free_blocks, free_count,
//  free_count_out, total_lens, token_offsets, slot_map, positions, block_size, seq_err, parent, stream)
PyObject* kv_plan_slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 17, [&] {
        const auto i32 = at::kInt;
        const at::Tensor& bt = ranked(a[3], "block_table", 2);
        const at::Tensor& pool = ranked(a[6], "free_blocks", 1);
        const at::Tensor& slots = ranked(a[11], "slot_map", 1);
        const int64_t B = bt.size(0), mb = bt.size(1), T = slots.size(0);
        const at::Tensor *lens = &tensor(a[1], "seq_lens"), *nl = &tensor(a[2], "new_lens"), *held = &tensor(a[4], "blocks_held"),
                         *ho = &tensor(a[5], "blocks_held_out"), *fc = &tensor(a[7], "free_count"), *fo = &tensor(a[8], "free_count_out"),
                         *tot = &tensor(a[9], "total_lens"), *off = &tensor(a[10], "token_offsets"), *pos = &tensor(a[12], "positions"),
                         *err = &tensor(a[14], "seq_err"), *par = a[15] == Py_None ? nullptr : &ranked(a[15], "parent", 2);
        auto p = [](void* x) { return static_cast<int32_t*>(x); };
        int32_t* p_bt = p(need(bt, "block_table", i32, {B, mb}));
        int32_t* p_pool = p(need(pool, "free_blocks", i32, {pool.size(0)}));
        auto* p_slots = static_cast<int64_t*>(need(slots, "slot_map", at::kLong, {T}));
        int32_t* p_pos = p(need(*pos, "positions", i32, {T}));
        int32_t* p_off = p(need(*off, "token_offsets", i32, {B + 1}));
        int32_t* p_lens = p(need(*lens, "seq_lens", i32, {B}));
        int32_t* p_nl = p(need(*nl, "new_lens", i32, {B}));
        int32_t* p_held = p(need(*held, "blocks_held", i32, {B}));
        int32_t* p_ho = p(need(*ho, "blocks_held_out", i32, {B}));
        int32_t* p_tot = p(need(*tot, "total_lens", i32, {B}));
        int32_t* p_err = p(need(*err, "seq_err", i32, {B}));
        int32_t* p_fc = p(need(*fc, "free_count", i32, {1}));
        int32_t* p_fo = p(need(*fo, "free_count_out", i32, {1}));
        const int64_t N = par ? par->size(1) : 0;
        int32_t* p_par = par ? p(need(*par, "parent", i32, {B, N})) : nullptr;
        const long bs = PyLong_AsLong(a[13]);
        if (bs == -1 && PyErr_Occurred()) return 0;
        void* s = stream_for(a[16], {lens, nl, par, &bt, held, ho, &pool, fc, fo, tot, off, &slots, pos, err});
        return call(entry<decltype(&tsv_kv_plan_slots)>(a[0]), p_lens, p_nl, p_par, p_bt, p_held, p_ho, p_pool, p_fc, p_fo, p_tot,
                    p_off, p_slots, p_pos, small(B, "B"), small(N, "N"), small(bs, "block_size"), small(mb, "max_blocks"),
                    small(pool.size(0), "num_blocks"), small(T, "max_tokens"), p_err, s);
    });
}

// The token stride, in elements, of [T, H, D] rows whose heads are contiguous.
int64_t token_rows(const at::Tensor& t, const char* name, at::ScalarType type, int64_t T, int64_t H, int64_t D) {
    const int64_t want[3] = {T, H, D};
    if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(want, 3) || t.stride(2) != 1 || (H > 1 && t.stride(1) != D))
        throw Refused(std::string(name) + " must be " + text(at::IntArrayRef(want, 3)) + " " + c10::toString(type) + " with contiguous heads");
    return T > 1 ? t.stride(0) : H * D;
}

// (entry, q, k, v, positions, inv_freq, q_out, k_cache, v_cache, slot_map, tok_err, sections, rounds,
//  neighbours, stream)
PyObject* rope_kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        const at::Tensor &q = ranked(a[1], "q", 3), &k = tensor(a[2], "k"), &v = tensor(a[3], "v"), &pos = tensor(a[4], "positions"),
                         &inv = ranked(a[5], "inv_freq", 1), &qo = tensor(a[6], "q_out"), &kc = ranked(a[7], "k_cache", 4),
                         &vc = tensor(a[8], "v_cache"), &slots = tensor(a[9], "slot_map"), &err = tensor(a[10], "tok_err");
        const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), nb = kc.size(0), bs = kc.size(1), Hkv = kc.size(2), half = inv.size(0);
        const at::ScalarType type = q.scalar_type();
        const tsv_dtype dt = dtype_of(q);
        if (pos.dim() != 1 && pos.dim() != 2) throw Refused("positions must be [T] or [axes, T]");
        const int64_t axes = pos.dim() == 2 ? pos.size(0) : 1;
        tsv_rope_options o{small(2 * half, "rotary_dim"), PyObject_IsTrue(a[13]), small(axes, "axes"), PyObject_IsTrue(a[12]), {0, 0, 0, 0}};
        if (a[11] == Py_None) {
            if (axes != 1) throw Refused("several position axes need their sections");
            o.sections[0] = small(half, "rotary_dim");
        } else {
            const Py_ssize_t ns = PySequence_Size(a[11]);
            if (ns < 0) return 0;
            if (ns != axes || ns > 4)
                throw Refused(std::to_string(ns) + " sections for " + std::to_string(axes) + " position axes (at most 4)");
            for (Py_ssize_t i = 0; i < ns; ++i) {
                PyObject* x = PySequence_GetItem(a[11], i);
                const long value = x ? PyLong_AsLong(x) : -1;
                Py_XDECREF(x);
                if (PyErr_Occurred()) return 0;
                if (value < 0 || value > half) throw Refused("a section must hold 0 to rotary_dim / 2 pairs");
                o.sections[i] = static_cast<int>(value);
            }
        }
        const int64_t qs = token_rows(q, "q", type, T, Hq, D), ks = token_rows(k, "k", type, T, Hkv, D),
                      vs = token_rows(v, "v", type, T, Hkv, D), qos = token_rows(qo, "q_out", type, T, Hq, D);
        void* p_kc = need(kc, "k_cache", type, {nb, bs, Hkv, D});
        void* p_vc = need(vc, "v_cache", type, {nb, bs, Hkv, D});
        auto* p_pos = static_cast<int32_t*>(pos.dim() == 2 ? need(pos, "positions", at::kInt, {axes, T}) : need(pos, "positions", at::kInt, {T}));
        auto* p_inv = static_cast<float*>(need(inv, "inv_freq", at::kFloat, {half}));
        auto* p_slots = static_cast<int64_t*>(need(slots, "slot_map", at::kLong, {T}));
        auto* p_err = static_cast<int32_t*>(need(err, "tok_err", at::kInt, {T}));
        void* s = stream_for(a[14], {&q, &k, &v, &pos, &inv, &qo, &kc, &vc, &slots, &err});
        return call(entry<decltype(&tsv_rope_kv_append)>(a[0]), q.data_ptr(), k.data_ptr(), v.data_ptr(), p_pos, p_inv, qo.data_ptr(),
                    p_kc, p_vc, p_slots, small(T, "T"), small(Hq, "Hq"), small(Hkv, "Hkv"), small(D, "D"), qs, ks, vs, qos,
                    small(bs, "block_size"), small(nb, "num_blocks"), dt, &o, p_err, s);
    });
}

// (entry, q, k_cache, v_cache, block_table, seq_lens, out, scale, workspace, seq_err, lse, stream)
PyObject* decode_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        const at::Tensor &q = ranked(a[1], "q", 3), &kc = ranked(a[2], "k_cache", 4), &vc = tensor(a[3], "v_cache"),
                         &bt = ranked(a[4], "block_table", 2), &lens = tensor(a[5], "seq_lens"), &out = tensor(a[6], "out"),
                         &err = tensor(a[9], "seq_err");
        const at::Tensor *ws = a[8] == Py_None ? nullptr : &tensor(a[8], "workspace"), *lse = a[10] == Py_None ? nullptr : &tensor(a[10], "lse");
        const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2), nb = kc.size(0), bs = kc.size(1), Hkv = kc.size(2), mb = bt.size(1);
        const at::ScalarType type = q.scalar_type();
        const tsv_dtype dt = dtype_of(q);
        void* p_q = need(q, "q", type, {B, Hq, D});
        void* p_out = need(out, "out", type, {B, Hq, D});
        void* p_kc = need(kc, "k_cache", type, {nb, bs, Hkv, D});
        void* p_vc = need(vc, "v_cache", type, {nb, bs, Hkv, D});
        auto* p_bt = static_cast<int32_t*>(need(bt, "block_table", at::kInt, {B, mb}));
        auto* p_lens = static_cast<int32_t*>(need(lens, "seq_lens", at::kInt, {B}));
        auto* p_err = static_cast<int32_t*>(need(err, "seq_err", at::kInt, {B}));
        auto* p_lse = lse ? static_cast<float*>(need(*lse, "lse", at::kFloat, {B, Hq})) : nullptr;
        if (ws && !ws->is_contiguous()) throw Refused("workspace must be contiguous");
        const double scale = PyFloat_AsDouble(a[7]);
        if (scale == -1.0 && PyErr_Occurred()) return 0;
        void* s = stream_for(a[11], {&q, &kc, &vc, &bt, &lens, &out, ws, &err, lse});
        return call(entry<decltype(&tsv_decode_attn)>(a[0]), p_q, p_kc, p_vc, p_bt, p_lens, p_out, p_lse, small(B, "B"), small(Hq, "Hq"),
                    small(Hkv, "Hkv"), small(D, "D"), small(bs, "block_size"), small(mb, "max_blocks"), small(nb, "num_blocks"),
                    static_cast<float>(scale), dt, ws ? ws->data_ptr() : nullptr, ws ? ws->nbytes() : size_t(0), p_err, s);
    });
}

PyMethodDef methods[] = {
    {"kv_plan_slots", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_plan_slots)), METH_FASTCALL, nullptr},
    {"rope_kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_kv_append)), METH_FASTCALL, nullptr},
    {"decode_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode_attn)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
