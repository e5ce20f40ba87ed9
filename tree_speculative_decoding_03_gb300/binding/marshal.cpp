// marshal.cpp -- argument marshalling of the serving operators: torch tensors to the C ABI.
//
// A decoding step calls these operators once per layer or step, each on up to sixteen
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

int32_t* ints(const at::Tensor& t, const char* name, int64_t n) { return static_cast<int32_t*>(need(t, name, at::kInt, {n})); }

// (entry, fork_src, fork_dst, seq_lens, seq_lens_out, block_table, blocks_held, blocks_held_out, shares, shares_out, free_blocks,
//  free_count, free_count_out, copy_src, copy_dst, copy_rows, block_size, fork_err, stream)
PyObject* kv_fork_seqs(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 19, [&] {
        const at::Tensor &fs = ranked(a[1], "fork_src", 1), &fd = tensor(a[2], "fork_dst"), &lens = tensor(a[3], "seq_lens"),
                         &lo = tensor(a[4], "seq_lens_out"), &bt = ranked(a[5], "block_table", 2), &held = tensor(a[6], "blocks_held"),
                         &ho = tensor(a[7], "blocks_held_out"), &sh = ranked(a[8], "shares", 1), &so = tensor(a[9], "shares_out"),
                         &pool = tensor(a[10], "free_blocks"), &fc = tensor(a[11], "free_count"), &fo = tensor(a[12], "free_count_out"),
                         &cs = tensor(a[13], "copy_src"), &cd = tensor(a[14], "copy_dst"), &cr = tensor(a[15], "copy_rows"),
                         &err = tensor(a[17], "fork_err");
        const int64_t F = fs.size(0), B = bt.size(0), mb = bt.size(1), nb = sh.size(0);
        auto* p_bt = static_cast<int32_t*>(need(bt, "block_table", at::kInt, {B, mb}));
        int32_t *p_fs = ints(fs, "fork_src", F), *p_fd = ints(fd, "fork_dst", F), *p_lens = ints(lens, "seq_lens", B),
                *p_lo = ints(lo, "seq_lens_out", B), *p_held = ints(held, "blocks_held", B), *p_ho = ints(ho, "blocks_held_out", B),
                *p_sh = ints(sh, "shares", nb), *p_so = ints(so, "shares_out", nb), *p_pool = ints(pool, "free_blocks", nb),
                *p_fc = ints(fc, "free_count", 1), *p_fo = ints(fo, "free_count_out", 1), *p_cs = ints(cs, "copy_src", F),
                *p_cd = ints(cd, "copy_dst", F), *p_cr = ints(cr, "copy_rows", F), *p_err = ints(err, "fork_err", F);
        const long bs = PyLong_AsLong(a[16]);
        if (bs == -1 && PyErr_Occurred()) return 0;
        void* s = stream_for(a[18], {&bt, &fs, &fd, &lens, &lo, &held, &ho, &sh, &so, &pool, &fc, &fo, &cs, &cd, &cr, &err});
        return call(entry<decltype(&tsv_kv_fork_seqs)>(a[0]), p_fs, p_fd, p_lens, p_lo, p_bt, p_held, p_ho, p_sh, p_so, p_pool, p_fc, p_fo,
                    p_cs, p_cd, p_cr, small(F, "F"), small(B, "B"), small(bs, "block_size"), small(mb, "max_blocks"),
                    small(nb, "num_blocks"), p_err, s);
    });
}

// (entry, keep_lens, block_table, blocks_held, blocks_held_out, shares, shares_out, free_blocks, free_count, free_count_out, block_size,
//  seq_err, stream)
PyObject* kv_release_seqs(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        const at::Tensor &keep = tensor(a[1], "keep_lens"), &bt = ranked(a[2], "block_table", 2), &held = tensor(a[3], "blocks_held"),
                         &ho = tensor(a[4], "blocks_held_out"), &sh = ranked(a[5], "shares", 1), &so = tensor(a[6], "shares_out"),
                         &pool = tensor(a[7], "free_blocks"), &fc = tensor(a[8], "free_count"), &fo = tensor(a[9], "free_count_out"),
                         &err = tensor(a[11], "seq_err");
        const int64_t B = bt.size(0), mb = bt.size(1), nb = sh.size(0);
        auto* p_bt = static_cast<int32_t*>(need(bt, "block_table", at::kInt, {B, mb}));
        int32_t *p_keep = ints(keep, "keep_lens", B), *p_held = ints(held, "blocks_held", B), *p_ho = ints(ho, "blocks_held_out", B),
                *p_sh = ints(sh, "shares", nb), *p_so = ints(so, "shares_out", nb), *p_pool = ints(pool, "free_blocks", nb),
                *p_fc = ints(fc, "free_count", 1), *p_fo = ints(fo, "free_count_out", 1), *p_err = ints(err, "seq_err", B);
        const long bs = PyLong_AsLong(a[10]);
        if (bs == -1 && PyErr_Occurred()) return 0;
        void* s = stream_for(a[12], {&bt, &keep, &held, &ho, &sh, &so, &pool, &fc, &fo, &err});
        return call(entry<decltype(&tsv_kv_release_seqs)>(a[0]), p_keep, p_bt, p_held, p_ho, p_sh, p_so, p_pool, p_fc, p_fo, small(B, "B"),
                    small(bs, "block_size"), small(mb, "max_blocks"), small(nb, "num_blocks"), p_err, s);
    });
}

// (entry, block_table, block_table_out, blocks_held, shares, shares_out, free_blocks, free_count_out, copy_src, copy_dst, copy_count,
//  seq_err, workspace, stream)
PyObject* kv_compact_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        const at::Tensor &bt = ranked(a[1], "block_table", 2), &bo = tensor(a[2], "block_table_out"), &held = tensor(a[3], "blocks_held"),
                         &sh = ranked(a[4], "shares", 1), &so = tensor(a[5], "shares_out"), &pool = tensor(a[6], "free_blocks"),
                         &fo = tensor(a[7], "free_count_out"), &cs = tensor(a[8], "copy_src"), &cd = tensor(a[9], "copy_dst"),
                         &cc = tensor(a[10], "copy_count"), &err = tensor(a[11], "seq_err"), &ws = tensor(a[12], "workspace");
        const int64_t B = bt.size(0), mb = bt.size(1), nb = sh.size(0);
        auto* p_bt = static_cast<int32_t*>(need(bt, "block_table", at::kInt, {B, mb}));
        auto* p_bo = static_cast<int32_t*>(need(bo, "block_table_out", at::kInt, {B, mb}));
        int32_t *p_held = ints(held, "blocks_held", B), *p_sh = ints(sh, "shares", nb), *p_so = ints(so, "shares_out", nb),
                *p_pool = ints(pool, "free_blocks", nb), *p_fo = ints(fo, "free_count_out", 1), *p_cs = ints(cs, "copy_src", nb / 2),
                *p_cd = ints(cd, "copy_dst", nb / 2), *p_cc = ints(cc, "copy_count", 1), *p_err = ints(err, "seq_err", B);
        if (!ws.is_contiguous()) throw Refused("workspace must be contiguous");
        void* s = stream_for(a[13], {&bt, &bo, &held, &sh, &so, &pool, &fo, &cs, &cd, &cc, &err, &ws});
        return call(entry<decltype(&tsv_kv_compact_blocks)>(a[0]), p_bt, p_bo, p_held, p_sh, p_so, p_pool, p_fo, p_cs, p_cd, p_cc,
                    small(B, "B"), small(mb, "max_blocks"), small(nb, "num_blocks"), ws.data_ptr(), ws.nbytes(), p_err, s);
    });
}

// (entry, k_cache, v_cache, copy_src, copy_dst, copy_rows, copy_count, copy_err, stream)
PyObject* kv_copy_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const at::Tensor &kc = ranked(a[1], "k_cache", 4), &vc = tensor(a[2], "v_cache"), &cs = ranked(a[3], "copy_src", 1),
                         &cd = tensor(a[4], "copy_dst"), &err = tensor(a[7], "copy_err");
        const at::Tensor *rows = a[5] == Py_None ? nullptr : &tensor(a[5], "copy_rows"), *count = a[6] == Py_None ? nullptr : &tensor(a[6], "copy_count");
        const int64_t m = cs.size(0), nb = kc.size(0), bs = kc.size(1), Hkv = kc.size(2), D = kc.size(3);
        const tsv_dtype dt = dtype_of(kc);
        void* p_kc = need(kc, "k_cache", kc.scalar_type(), {nb, bs, Hkv, D});
        void* p_vc = need(vc, "v_cache", kc.scalar_type(), {nb, bs, Hkv, D});
        int32_t *p_cs = ints(cs, "copy_src", m), *p_cd = ints(cd, "copy_dst", m), *p_err = ints(err, "copy_err", m),
                *p_rows = rows ? ints(*rows, "copy_rows", m) : nullptr, *p_count = count ? ints(*count, "copy_count", 1) : nullptr;
        void* s = stream_for(a[8], {&kc, &vc, &cs, &cd, rows, count, &err});
        return call(entry<decltype(&tsv_kv_copy_blocks)>(a[0]), p_kc, p_vc, p_cs, p_cd, p_rows, p_count, small(m, "n"), small(Hkv, "Hkv"),
                    small(D, "D"), small(bs, "block_size"), small(nb, "num_blocks"), dt, p_err, s);
    });
}

// (entry, q, k_cache, v_cache, block_table, seq_lens, group_offsets, prefix_lens, out, scale, workspace, seq_err, lse, stream)
PyObject* prefix_decode_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        const at::Tensor &q = ranked(a[1], "q", 3), &kc = ranked(a[2], "k_cache", 4), &vc = tensor(a[3], "v_cache"),
                         &bt = ranked(a[4], "block_table", 2), &lens = tensor(a[5], "seq_lens"), &off = tensor(a[6], "group_offsets"),
                         &pre = ranked(a[7], "prefix_lens", 1), &out = tensor(a[8], "out"), &err = tensor(a[11], "seq_err");
        const at::Tensor *ws = a[10] == Py_None ? nullptr : &tensor(a[10], "workspace"), *lse = a[12] == Py_None ? nullptr : &tensor(a[12], "lse");
        const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2), nb = kc.size(0), bs = kc.size(1), Hkv = kc.size(2), mb = bt.size(1),
                      G = pre.size(0);
        const at::ScalarType type = q.scalar_type();
        const tsv_dtype dt = dtype_of(q);
        void* p_q = need(q, "q", type, {B, Hq, D});
        void* p_out = need(out, "out", type, {B, Hq, D});
        void* p_kc = need(kc, "k_cache", type, {nb, bs, Hkv, D});
        void* p_vc = need(vc, "v_cache", type, {nb, bs, Hkv, D});
        auto* p_bt = static_cast<int32_t*>(need(bt, "block_table", at::kInt, {B, mb}));
        int32_t *p_lens = ints(lens, "seq_lens", B), *p_off = ints(off, "group_offsets", G + 1), *p_pre = ints(pre, "prefix_lens", G),
                *p_err = ints(err, "seq_err", B);
        auto* p_lse = lse ? static_cast<float*>(need(*lse, "lse", at::kFloat, {B, Hq})) : nullptr;
        if (ws && !ws->is_contiguous()) throw Refused("workspace must be contiguous");
        const double scale = PyFloat_AsDouble(a[9]);
        if (scale == -1.0 && PyErr_Occurred()) return 0;
        void* s = stream_for(a[13], {&q, &kc, &vc, &bt, &lens, &off, &pre, &out, ws, &err, lse});
        return call(entry<decltype(&tsv_prefix_decode_attn)>(a[0]), p_q, p_kc, p_vc, p_bt, p_lens, p_off, p_pre, p_out, p_lse, small(B, "B"),
                    small(G, "G"), small(Hq, "Hq"), small(Hkv, "Hkv"), small(D, "D"), small(bs, "block_size"), small(mb, "max_blocks"),
                    small(nb, "num_blocks"), static_cast<float>(scale), dt, ws ? ws->data_ptr() : nullptr, ws ? ws->nbytes() : size_t(0), p_err, s);
    });
}

// (entry, logits, tokens, logprobs, tok_err, temperature, entropy, top_ids, top_logprobs, stream)
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const at::Tensor &x = ranked(a[1], "logits", 2), &tok = tensor(a[2], "tokens"), &lp = tensor(a[3], "logprobs"), &err = tensor(a[4], "tok_err");
        const at::Tensor *ent = a[6] == Py_None ? nullptr : &tensor(a[6], "entropy"), *ids = a[7] == Py_None ? nullptr : &ranked(a[7], "top_ids", 2),
                         *tops = a[8] == Py_None ? nullptr : &tensor(a[8], "top_logprobs");
        const int64_t T = x.size(0), V = x.size(1), top = ids ? ids->size(1) : 0;
        const tsv_dtype dt = dtype_of(x);
        if (V > 1 && x.stride(1) != 1) throw Refused("logits must have contiguous rows");
        if ((ids == nullptr) != (tops == nullptr)) throw Refused("top_ids and top_logprobs go together");
        int32_t *p_tok = ints(tok, "tokens", T), *p_err = ints(err, "tok_err", T);
        auto* p_lp = static_cast<float*>(need(lp, "logprobs", at::kFloat, {T}));
        auto* p_ent = ent ? static_cast<float*>(need(*ent, "entropy", at::kFloat, {T})) : nullptr;
        auto* p_ids = ids ? static_cast<int32_t*>(need(*ids, "top_ids", at::kInt, {T, top})) : nullptr;
        auto* p_tops = tops ? static_cast<float*>(need(*tops, "top_logprobs", at::kFloat, {T, top})) : nullptr;
        const double temp = PyFloat_AsDouble(a[5]);
        if (temp == -1.0 && PyErr_Occurred()) return 0;
        void* s = stream_for(a[9], {&x, &tok, &lp, &err, ent, ids, tops});
        return call(entry<decltype(&tsv_token_logprobs)>(a[0]), x.data_ptr(), T > 1 ? x.stride(0) : V, p_tok, small(T, "T"), small(V, "V"),
                    static_cast<float>(temp), small(top, "top"), dt, p_lp, p_ent, p_ids, p_tops, p_err, s);
    });
}

PyMethodDef methods[] = {
    {"kv_fork_seqs", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_fork_seqs)), METH_FASTCALL, nullptr},
    {"kv_release_seqs", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_release_seqs)), METH_FASTCALL, nullptr},
    {"kv_compact_blocks", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_compact_blocks)), METH_FASTCALL, nullptr},
    {"kv_copy_blocks", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_copy_blocks)), METH_FASTCALL, nullptr},
    {"prefix_decode_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefix_decode_attn)), METH_FASTCALL, nullptr},
    {"token_logprobs", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(token_logprobs)), METH_FASTCALL, nullptr},
    {"kv_plan_slots", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_plan_slots)), METH_FASTCALL, nullptr},
    {"rope_kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_kv_append)), METH_FASTCALL, nullptr},
    {"decode_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode_attn)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
