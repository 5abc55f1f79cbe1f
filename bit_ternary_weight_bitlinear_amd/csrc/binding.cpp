// binding.cpp -- marshalling of the attention calls from torch tensors to the C
// ABI (include/bitlinear.h). One token's call runs a few microseconds on the
// device; looking at a dozen tensors from Python costs as much again (11 us for a
// decode call against 6.8 us on the device), so these calls check their tensors
// here. The library is the one the package has loaded: its functions are looked
// up by path at first use, and nothing here computes.
#include <Python.h>

#include <dlfcn.h>

#include <cmath>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/bitlinear.h"

namespace {

PyObject *g_error = nullptr;  // the package's exception class

struct Library {
    decltype(&bitlinear_status_string) status_string;
    decltype(&bitlinear_attention_workspace_size) attention_workspace_size;
    decltype(&bitlinear_attention) attention;
    decltype(&bitlinear_cache_append) cache_append;
    decltype(&bitlinear_cache_read) cache_read;
    decltype(&bitlinear_attention_cached_workspace_size) attention_cached_workspace_size;
    decltype(&bitlinear_attention_cached) attention_cached;
    decltype(&bitlinear_cache_evict) cache_evict;
    decltype(&bitlinear_rotate) rotate;
    decltype(&bitlinear_attention_shared_workspace_size) attention_shared_workspace_size;
    decltype(&bitlinear_attention_shared) attention_shared;
    decltype(&bitlinear_cache_bounds) cache_bounds;
    decltype(&bitlinear_block_select_workspace_size) block_select_workspace_size;
    decltype(&bitlinear_block_select) block_select;
    decltype(&bitlinear_attention_selected_workspace_size) attention_selected_workspace_size;
    decltype(&bitlinear_attention_selected) attention_selected;
} g_lib;

struct Refused {
    std::string what;
};
[[noreturn]] void refuse(const std::string &what) { throw Refused{what}; }

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}
std::string tensor_text(const at::Tensor &t)
{
    return std::string(c10::toString(t.scalar_type())) + " " + shape_text(t.sizes()) + " on " + t.device().str();
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a device (HIP) tensor");
    return THPVariable_Unpack(o);
}
// the first tensor of a call: names the device
const at::Tensor &first_tensor(PyObject *o, const char *name)
{
    const at::Tensor &t = tensor(o, name);
    if (!t.is_cuda()) refuse(std::string(name) + " must be a device (HIP) tensor");
    return t;
}

struct Rows {
    const void *p;
    int64_t stride, m, heads, d;
};
// q, k or v [m][heads][head_dim], a token's heads adjacent
Rows heads(const at::Tensor &t, const char *name, at::ScalarType type, at::Device device)
{
    if (t.scalar_type() != type || t.device() != device)
        refuse(std::string(name) + " must be " + c10::toString(type) + " on " + device.str() + ", got " + tensor_text(t));
    if (t.dim() != 3 || t.stride(2) != 1 || (t.stride(1) != t.size(2) && t.size(1) != 1))
        refuse(std::string(name) + " must be [m][heads][head_dim] with a token's heads adjacent");
    // the stride of a single token means nothing; torch may report any
    return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2), t.size(0), t.size(1), t.size(2)};
}

void *dense(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, at::Device device)
{
    if (t.scalar_type() != type || t.device() != device || t.sizes() != shape || !t.is_contiguous())
        refuse(std::string(name) + " must be " + c10::toString(type) + ", contiguous, of shape " + shape_text(shape) + " on " +
               device.str() + "; got " + tensor_text(t));
    return t.data_ptr();
}

bl_dtype act_dtype(at::ScalarType t)
{
    if (t == at::kFloat) return BL_F32;
    if (t == at::kBFloat16) return BL_BF16;
    refuse(std::string("activations must be float32 or bfloat16, got ") + c10::toString(t));
}

const int32_t *starts(PyObject *o, at::Device device, int64_t &seqs)
{
    const at::Tensor &t = tensor(o, "cu_seqlens");
    if (t.dim() != 1 || t.size(0) < 2) refuse("cu_seqlens must be int32 [seqs + 1]");
    seqs = t.size(0) - 1;
    return static_cast<const int32_t *>(dense(t, "cu_seqlens", at::kInt, t.sizes(), device));
}

struct Cache {
    int8_t *k, *v;
    float *ks, *vs;
    int64_t pages, heads, d;
};
// kv_heads, head_dim < 0: as the cache has them
Cache cache_args(PyObject *o, int64_t kv_heads, int64_t head_dim, at::Device device)
{
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) refuse("cache must be a KVCache");
    const at::Tensor &k = tensor(PyTuple_GET_ITEM(o, 0), "cache.k"), &v = tensor(PyTuple_GET_ITEM(o, 1), "cache.v");
    const at::Tensor &ks = tensor(PyTuple_GET_ITEM(o, 2), "cache.k_scale"), &vs = tensor(PyTuple_GET_ITEM(o, 3), "cache.v_scale");
    if (k.dim() != 3) refuse("cache.k must be int8 [pages][kv_heads][64 * head_dim]");
    const int64_t width = k.size(2) / BL_CACHE_BLOCK;
    if (k.size(2) % BL_CACHE_BLOCK || (head_dim >= 0 && width != head_dim) || (kv_heads >= 0 && k.size(1) != kv_heads))
        refuse("cache holds " + std::to_string(k.size(1)) + " heads of " + std::to_string(width) + ", not " +
               std::to_string(kv_heads >= 0 ? kv_heads : k.size(1)) + " of " + std::to_string(head_dim));
    const int64_t per[2] = {k.size(0), k.size(1)};
    return {static_cast<int8_t *>(dense(k, "cache.k", at::kChar, k.sizes(), device)),
            static_cast<int8_t *>(dense(v, "cache.v", at::kChar, k.sizes(), device)),
            static_cast<float *>(dense(ks, "cache.k_scale", at::kFloat, per, device)),
            static_cast<float *>(dense(vs, "cache.v_scale", at::kFloat, per, device)), k.size(0), k.size(1), width};
}

struct Table {
    const int32_t *cu, *lens, *table;
    int64_t seqs, wide;
};
Table table_args(PyObject *block_table, PyObject *lens, PyObject *cu, int64_t m, at::Device device, const char *name)
{
    Table r{};
    r.seqs = m;  // without cu_seqlens one row per sequence
    if (cu != Py_None) r.cu = starts(cu, device, r.seqs);
    const at::Tensor &t = tensor(block_table, "block_table");
    if (t.dim() != 2) refuse("block_table must be int32 [seqs][max_blocks]");
    r.wide = t.size(1);
    const int64_t per[1] = {r.seqs}, both[2] = {r.seqs, r.wide};
    r.lens = static_cast<const int32_t *>(dense(tensor(lens, name), name, at::kInt, per, device));
    r.table = static_cast<const int32_t *>(dense(t, "block_table", at::kInt, both, device));
    return r;
}

float scale_of(PyObject *o, int64_t d)
{
    if (o == Py_None) return (float)(1.0 / std::sqrt((double)d));
    const double v = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) refuse("");
    return (float)v;
}

int64_t int_of(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (PyErr_Occurred()) refuse("");
    return v;
}

// a caller's workspace, or undefined
at::Tensor given_workspace(PyObject *o) { return o == Py_None ? at::Tensor() : tensor(o, "workspace"); }

// A caller's workspace checked against the call's size, or one of the call's own.
// Runs without the interpreter's lock, so it sees no Python objects.
void *scratch(size_t bytes, at::Tensor &ws, at::Device device)
{
    if (bytes == 0) return nullptr;
    if (!ws.defined())
        ws = at::empty({(int64_t)bytes}, at::TensorOptions(at::kByte).device(device));
    else if (ws.device() != device || !ws.is_contiguous() || ws.nbytes() < bytes)
        refuse("workspace must be contiguous and hold " + std::to_string(bytes) + " bytes on " + device.str() + "; got " + tensor_text(ws));
    return ws.data_ptr();
}

// The caching allocator hands the memory of a call's own tensors on to later work
// of the same stream only, so they may end before the kernels do.
void *stream_of(at::Device device) { return c10::hip::getCurrentHIPStream(device.index()).stream(); }

void done(bl_status s, const char *what)
{
    if (s != BL_OK) refuse(std::string(what) + ": " + g_lib.status_string(s));
}

struct WithoutGil {
    PyThreadState *s = PyEval_SaveThread();
    ~WithoutGil() { PyEval_RestoreThread(s); }
};

// torch's own exception class
void out_of_memory(const char *what)
{
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, what);
    Py_XDECREF(type);
    Py_XDECREF(torch);
}

// No C++ exception leaves an entry
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f)
{
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused &r) {
        if (!PyErr_Occurred()) PyErr_SetString(g_error, r.what.c_str());
    } catch (const c10::OutOfMemoryError &e) {
        out_of_memory(e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

// (q, k, v, cu_seqlens, scale, out, workspace)
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 7, [&]() -> PyObject * {
        const at::Tensor &tq = first_tensor(a[0], "q");
        const at::Device device = tq.device();
        const at::ScalarType type = tq.scalar_type();
        const Rows q = heads(tq, "q", type, device), k = heads(tensor(a[1], "k"), "k", type, device),
                   v = heads(tensor(a[2], "v"), "v", type, device);
        if (k.m != q.m || v.m != q.m || k.d != q.d || v.d != q.d || k.heads != v.heads)
            refuse("k and v must be [" + std::to_string(q.m) + "][kv_heads][" + std::to_string(q.d) + "], got " +
                   shape_text(THPVariable_Unpack(a[1]).sizes()) + " and " + shape_text(THPVariable_Unpack(a[2]).sizes()));
        int64_t seqs;
        const int32_t *cu = starts(a[3], device, seqs);
        const bl_dtype dtype = act_dtype(type);
        const float scale = scale_of(a[4], q.d);
        const int64_t shape[2] = {q.m, q.heads * q.d};
        at::Tensor out, ws = given_workspace(a[6]);
        if (a[5] != Py_None) {
            out = tensor(a[5], "out");
            dense(out, "out", type, shape, device);
        }
        {
            WithoutGil free;
            const c10::DeviceGuard guard(device);
            if (!out.defined()) out = at::empty(shape, tq.options());
            const size_t bytes = g_lib.attention_workspace_size(dtype, q.m, q.heads, k.heads, q.d, seqs);
            void *const space = scratch(bytes, ws, device);
            done(g_lib.attention(q.p, q.stride, k.p, k.stride, v.p, v.stride, dtype, q.m, q.heads, k.heads, q.d, cu, seqs, scale,
                                 out.data_ptr(), space, bytes, stream_of(device)),
                 "bitlinear_attention");
        }
        return THPVariable_Wrap(out);
    });
}

// (cache, k, v, block_table, lens, cu_seqlens)
PyObject *cache_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&]() -> PyObject * {
        const at::Tensor &tk = first_tensor(a[1], "k");
        const at::Device device = tk.device();
        const at::ScalarType type = tk.scalar_type();
        const Rows k = heads(tk, "k", type, device), v = heads(tensor(a[2], "v"), "v", type, device);
        if (v.m != k.m || v.heads != k.heads || v.d != k.d)
            refuse("v must have shape " + shape_text(tk.sizes()) + ", got " + shape_text(THPVariable_Unpack(a[2]).sizes()));
        const bl_dtype dtype = act_dtype(type);
        const Cache c = cache_args(a[0], k.heads, k.d, device);
        const Table t = table_args(a[3], a[4], a[5], k.m, device, "lens");
        {
            WithoutGil free;
            const c10::DeviceGuard guard(device);
            done(g_lib.cache_append(k.p, k.stride, v.p, v.stride, dtype, k.m, k.heads, k.d, t.cu, t.lens, t.seqs, t.table, t.wide,
                                    c.k, c.v, c.ks, c.vs, c.pages, stream_of(device)),
                 "bitlinear_cache_append");
        }
        Py_RETURN_NONE;
    });
}

// (cache, block_table, begin, cu_seqlens, m, bf16)
PyObject *cache_read(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&]() -> PyObject * {
        if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 4) refuse("cache must be a KVCache");
        const at::Device device = first_tensor(PyTuple_GET_ITEM(a[0], 0), "cache.k").device();
        const Cache c = cache_args(a[0], -1, -1, device);
        const int64_t m = int_of(a[4]);
        const bool bf16 = PyObject_IsTrue(a[5]) == 1;
        const Table t = table_args(a[1], a[2], a[3], m, device, "begin");
        if (m < 1) done(BL_ERR_SHAPE, "bitlinear_cache_read");
        at::Tensor k, v;
        {
            WithoutGil free;
            const c10::DeviceGuard guard(device);
            k = at::empty({m, c.heads, c.d}, at::TensorOptions(bf16 ? at::kBFloat16 : at::kFloat).device(device));
            v = at::empty_like(k);
            done(g_lib.cache_read(c.k, c.v, c.ks, c.vs, c.pages, t.table, t.wide, t.cu, t.lens, t.seqs, bf16 ? BL_BF16 : BL_F32, m,
                                  c.heads, c.d, k.data_ptr(), v.data_ptr(), stream_of(device)),
                 "bitlinear_cache_read");
        }
        return Py_BuildValue("NN", THPVariable_Wrap(k), THPVariable_Wrap(v));
    });
}

// (q, cache, block_table, lens, cu_seqlens, scale, weights, out, workspace)
PyObject *attention_cached(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 9, [&]() -> PyObject * {
        const at::Tensor &tq = first_tensor(a[0], "q");
        const at::Device device = tq.device();
        const at::ScalarType type = tq.scalar_type();
        const Rows q = heads(tq, "q", type, device);
        const bl_dtype dtype = act_dtype(type);
        const Cache c = cache_args(a[1], -1, q.d, device);
        const Table t = table_args(a[2], a[3], a[4], q.m, device, "lens");
        const float scale = scale_of(a[5], q.d);
        float *weights = nullptr;
        if (a[6] != Py_None) {
            const int64_t both[2] = {t.seqs, t.wide};
            weights = static_cast<float *>(dense(tensor(a[6], "weights"), "weights", at::kFloat, both, device));
        }
        const int64_t shape[2] = {q.m, q.heads * q.d};
        at::Tensor out, ws = given_workspace(a[8]);
        if (a[7] != Py_None) {
            out = tensor(a[7], "out");
            dense(out, "out", type, shape, device);
        }
        {
            WithoutGil free;
            const c10::DeviceGuard guard(device);
            if (!out.defined()) out = at::empty(shape, tq.options());
            const size_t bytes =
                g_lib.attention_cached_workspace_size(q.m, q.heads, c.heads, q.d, t.seqs, t.wide, weights != nullptr);
            void *const space = scratch(bytes, ws, device);
            done(g_lib.attention_cached(q.p, q.stride, dtype, q.m, q.heads, c.heads, q.d, t.cu, t.lens, t.seqs, t.table, t.wide, c.k,
                                        c.v, c.ks, c.vs, c.pages, scale, out.data_ptr(), weights, space,
                                        bytes, stream_of(device)),
                 "bitlinear_attention_cached");
        }
        return THPVariable_Wrap(out);
    });
}

// (block_table, lens, weights, keep, first, recent)
PyObject *cache_evict(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&]() -> PyObject * {
        const at::Tensor &table = first_tensor(a[0], "block_table");
        const at::Device device = table.device();
        if (table.dim() != 2) refuse("block_table must be int32 [seqs][max_blocks]");
        const int64_t seqs = table.size(0), wide = table.size(1), per[1] = {seqs}, both[2] = {seqs, wide};
        const at::Tensor &lens = tensor(a[1], "lens"), &weights = tensor(a[2], "weights");
        const auto *tp = static_cast<const int32_t *>(dense(table, "block_table", at::kInt, both, device));
        const auto *lp = static_cast<const int32_t *>(dense(lens, "lens", at::kInt, per, device));
        const auto *wp = static_cast<const float *>(dense(weights, "weights", at::kFloat, both, device));
        const int64_t keep = int_of(a[3]), first = int_of(a[4]), recent = int_of(a[5]);
        at::Tensor t2, l2, w2, gone, count;
        {
            WithoutGil free;
            const c10::DeviceGuard guard(device);
            t2 = at::empty(both, table.options());
            gone = at::empty(both, table.options());
            l2 = at::empty(per, lens.options());
            count = at::empty(per, lens.options());
            w2 = at::empty(both, weights.options());
            done(g_lib.cache_evict(tp, lp, wp, seqs, wide, keep, first, recent, static_cast<int32_t *>(t2.data_ptr()),
                                   static_cast<int32_t *>(l2.data_ptr()), static_cast<float *>(w2.data_ptr()),
                                   static_cast<int32_t *>(gone.data_ptr()), static_cast<int32_t *>(count.data_ptr()),
                                   stream_of(device)),
                 "bitlinear_cache_evict");
        }
        return Py_BuildValue("NNNNN", THPVariable_Wrap(t2), THPVariable_Wrap(l2), THPVariable_Wrap(w2), THPVariable_Wrap(gone),
                             THPVariable_Wrap(count));
    });
}

// an optional gain of every head's norm
const float *gain_of(PyObject *o, const char *name, int64_t d, at::Device device)
{
    if (o == Py_None) return nullptr;
    const int64_t per[1] = {d};
    return static_cast<const float *>(dense(tensor(o, name), name, at::kFloat, per, device));
}

float float_of(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) refuse("");
    return (float)v;
}

// (q, k, inv_freq, begin, cu_seqlens, interleaved, q_gain, k_gain, eps, magnitude, out)
PyObject *rotate(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [&]() -> PyObject * {
        const at::Tensor &tq = first_tensor(a[0], "q"), &tk = tensor(a[1], "k");
        const at::Device device = tq.device();
        const at::ScalarType type = tq.scalar_type();
        const Rows q = heads(tq, "q", type, device), k = heads(tk, "k", type, device);
        const bl_dtype dtype = act_dtype(type);
        if (k.m != q.m || k.d != q.d)
            refuse("k must be [" + std::to_string(q.m) + "][kv_heads][" + std::to_string(q.d) + "], got " + shape_text(tk.sizes()));
        const at::Tensor &freq = tensor(a[2], "inv_freq");
        const auto *fp = static_cast<const float *>(dense(freq, "inv_freq", at::kFloat, freq.sizes(), device));
        if (freq.dim() != 1) refuse("inv_freq must be fp32 [rotary_dim / 2]");
        int64_t seqs = q.m;
        const int32_t *cu = a[4] == Py_None ? nullptr : starts(a[4], device, seqs);
        const int64_t per[1] = {seqs};
        const auto *begin = static_cast<const int32_t *>(dense(tensor(a[3], "begin"), "begin", at::kInt, per, device));
        const int interleaved = PyObject_IsTrue(a[5]);
        if (interleaved < 0) refuse("");
        const float *gq = gain_of(a[6], "q_gain", q.d, device), *gk = gain_of(a[7], "k_gain", q.d, device);
        const float eps = float_of(a[8]), magnitude = float_of(a[9]);
        at::Tensor oq, ok;
        Rows q2 = q, k2 = k;
        if (a[10] != Py_None) {
            if (!PyTuple_Check(a[10]) || PyTuple_GET_SIZE(a[10]) != 2) refuse("out must be two tensors");
            oq = tensor(PyTuple_GET_ITEM(a[10], 0), "out[0]");
            ok = tensor(PyTuple_GET_ITEM(a[10], 1), "out[1]");
            q2 = heads(oq, "out[0]", type, device);
            k2 = heads(ok, "out[1]", type, device);
            if (oq.sizes() != tq.sizes() || ok.sizes() != tk.sizes())
                refuse("out must have the shapes of q and k, got " + shape_text(oq.sizes()) + " and " + shape_text(ok.sizes()));
        }
        {
            WithoutGil free;
            const c10::DeviceGuard guard(device);
            if (!oq.defined()) {
                oq = at::empty(tq.sizes(), tq.options());
                ok = at::empty(tk.sizes(), tk.options());
                q2 = {oq.data_ptr(), q.heads * q.d, q.m, q.heads, q.d};
                k2 = {ok.data_ptr(), k.heads * k.d, k.m, k.heads, k.d};
            }
            done(g_lib.rotate(q.p, q.stride, k.p, k.stride, dtype, q.m, q.heads, k.heads, q.d, cu, begin, seqs, fp, 2 * freq.size(0),
                              interleaved, magnitude, gq, gk, eps, const_cast<void *>(q2.p), q2.stride, const_cast<void *>(k2.p),
                              k2.stride, stream_of(device)),
                 "bitlinear_rotate");
        }
        return Py_BuildValue("NN", THPVariable_Wrap(oq), THPVariable_Wrap(ok));
    });
}

// (q, cache, prefix_table, prefix_len, block_table, lens, cu_seqlens, scale, out, workspace)
PyObject *attention_shared(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 10, [&]() -> PyObject * {
        const at::Tensor &tq = first_tensor(a[0], "q");
        const at::Device device = tq.device();
        const at::ScalarType type = tq.scalar_type();
        const Rows q = heads(tq, "q", type, device);
        const bl_dtype dtype = act_dtype(type);
        const Cache c = cache_args(a[1], -1, q.d, device);
        const at::Tensor &pt = tensor(a[2], "prefix_table");
        if (pt.dim() != 1) refuse("prefix_table must be int32 [prefix_blocks]");
        const auto *pages = static_cast<const int32_t *>(dense(pt, "prefix_table", at::kInt, pt.sizes(), device));
        const int64_t one[1] = {1};
        const auto *length = static_cast<const int32_t *>(dense(tensor(a[3], "prefix_len"), "prefix_len", at::kInt, one, device));
        const Table t = table_args(a[4], a[5], a[6], q.m, device, "lens");
        const float scale = scale_of(a[7], q.d);
        const int64_t shape[2] = {q.m, q.heads * q.d};
        at::Tensor out, ws = given_workspace(a[9]);
        if (a[8] != Py_None) {
            out = tensor(a[8], "out");
            dense(out, "out", type, shape, device);
        }
        {
            WithoutGil free;
            const c10::DeviceGuard guard(device);
            if (!out.defined()) out = at::empty(shape, tq.options());
            const size_t bytes = g_lib.attention_shared_workspace_size(q.m, q.heads, c.heads, q.d, t.seqs, t.wide, pt.size(0));
            void *const space = scratch(bytes, ws, device);
            done(g_lib.attention_shared(q.p, q.stride, dtype, q.m, q.heads, c.heads, q.d, pages, pt.size(0), length, t.cu, t.lens,
                                        t.seqs, t.table, t.wide, c.k, c.v, c.ks, c.vs, c.pages, scale, out.data_ptr(), space, bytes,
                                        stream_of(device)),
                 "bitlinear_attention_shared");
        }
        return THPVariable_Wrap(out);
    });
}

struct Bounds {
    int8_t *p;
    int64_t pages, heads, d;
};
Bounds bounds_of(PyObject *o, at::Device device)
{
    const at::Tensor &t = tensor(o, "bounds");
    if (t.dim() != 4 || t.size(2) != 2) refuse("bounds must be int8 [pages][kv_heads][2][head_dim]");
    return {static_cast<int8_t *>(dense(t, "bounds", at::kChar, t.sizes(), device)), t.size(0), t.size(1), t.size(3)};
}

// (cache, bounds, block_table, lens, cu_seqlens, m)
PyObject *cache_bounds(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&]() -> PyObject * {
        if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 4) refuse("cache must be a KVCache");
        const at::Device device = first_tensor(PyTuple_GET_ITEM(a[0], 0), "cache.k").device();
        const Cache c = cache_args(a[0], -1, -1, device);
        const Bounds b = bounds_of(a[1], device);
        if (b.pages != c.pages || b.heads != c.heads || b.d != c.d)
            refuse("bounds must be [" + std::to_string(c.pages) + "][" + std::to_string(c.heads) + "][2][" + std::to_string(c.d) +
                   "], got " + shape_text(THPVariable_Unpack(a[1]).sizes()));
        const int64_t m = int_of(a[5]);
        const Table t = table_args(a[2], a[3], a[4], m, device, "lens");
        {
            WithoutGil free;
            const c10::DeviceGuard guard(device);
            done(g_lib.cache_bounds(c.k, c.pages, c.heads, c.d, m, t.cu, t.lens, t.seqs, t.table, t.wide, b.p, stream_of(device)),
                 "bitlinear_cache_bounds");
        }
        Py_RETURN_NONE;
    });
}

// (q, bounds, k_scale, block_table, lens, keep, cu_seqlens, first, recent, out, workspace)
PyObject *block_select(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [&]() -> PyObject * {
        const at::Tensor &tq = first_tensor(a[0], "q");
        const at::Device device = tq.device();
        const at::ScalarType type = tq.scalar_type();
        const Rows q = heads(tq, "q", type, device);
        const bl_dtype dtype = act_dtype(type);
        const Bounds b = bounds_of(a[1], device);
        if (b.d != q.d) refuse("bounds are of heads of " + std::to_string(b.d) + ", q of " + std::to_string(q.d));
        const int64_t per[2] = {b.pages, b.heads};
        const auto *ks = static_cast<const float *>(dense(tensor(a[2], "k_scale"), "k_scale", at::kFloat, per, device));
        const Table t = table_args(a[3], a[4], a[6], q.m, device, "lens");
        const int64_t keep = int_of(a[5]), first = int_of(a[7]), recent = int_of(a[8]);
        // before there is an output of that size
        if (keep < 1 || keep > BL_MAX_DIM) done(BL_ERR_VALUE, "bitlinear_block_select");
        const int64_t shape[3] = {q.m, b.heads, keep};
        at::Tensor out, ws = given_workspace(a[10]);
        if (a[9] != Py_None) {
            out = tensor(a[9], "out");
            dense(out, "out", at::kInt, shape, device);
        }
        {
            WithoutGil free;
            const c10::DeviceGuard guard(device);
            if (!out.defined()) out = at::empty(shape, at::TensorOptions(at::kInt).device(device));
            const size_t bytes = g_lib.block_select_workspace_size(q.m, b.heads, t.wide);
            void *const space = scratch(bytes, ws, device);
            done(g_lib.block_select(q.p, q.stride, dtype, q.m, q.heads, b.heads, q.d, t.cu, t.lens, t.seqs, t.table, t.wide, b.p, ks,
                                    b.pages, keep, first, recent, static_cast<int32_t *>(out.data_ptr()), space, bytes,
                                    stream_of(device)),
                 "bitlinear_block_select");
        }
        return THPVariable_Wrap(out);
    });
}

// (q, cache, block_table, lens, selected, cu_seqlens, scale, out, workspace)
PyObject *attention_selected(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 9, [&]() -> PyObject * {
        const at::Tensor &tq = first_tensor(a[0], "q");
        const at::Device device = tq.device();
        const at::ScalarType type = tq.scalar_type();
        const Rows q = heads(tq, "q", type, device);
        const bl_dtype dtype = act_dtype(type);
        const Cache c = cache_args(a[1], -1, q.d, device);
        const Table t = table_args(a[2], a[3], a[5], q.m, device, "lens");
        const at::Tensor &sel = tensor(a[4], "selected");
        if (sel.dim() != 3) refuse("selected must be int32 [m][kv_heads][keep]");
        const int64_t each[3] = {q.m, c.heads, sel.size(2)};
        const auto *chosen = static_cast<const int32_t *>(dense(sel, "selected", at::kInt, each, device));
        const float scale = scale_of(a[6], q.d);
        const int64_t shape[2] = {q.m, q.heads * q.d};
        at::Tensor out, ws = given_workspace(a[8]);
        if (a[7] != Py_None) {
            out = tensor(a[7], "out");
            dense(out, "out", type, shape, device);
        }
        {
            WithoutGil free;
            const c10::DeviceGuard guard(device);
            if (!out.defined()) out = at::empty(shape, tq.options());
            const size_t bytes = g_lib.attention_selected_workspace_size(q.m, q.heads, c.heads, q.d, each[2]);
            void *const space = scratch(bytes, ws, device);
            done(g_lib.attention_selected(q.p, q.stride, dtype, q.m, q.heads, c.heads, q.d, t.cu, t.lens, t.seqs, t.table, t.wide, chosen,
                                          each[2], c.k, c.v, c.ks, c.vs, c.pages, scale, out.data_ptr(), space, bytes,
                                          stream_of(device)),
                 "bitlinear_attention_selected");
        }
        return THPVariable_Wrap(out);
    });
}

template <typename F>
bool find(void *lib, const char *name, F &f)
{
    f = reinterpret_cast<F>(dlsym(lib, name));
    return f != nullptr;
}

// (path of libbitlinear.so, exception class)
PyObject *bind(PyObject *, PyObject *args)
{
    const char *path;
    PyObject *error;
    if (!PyArg_ParseTuple(args, "sO", &path, &error)) return nullptr;
    void *lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    Library l;
    if (!lib || !find(lib, "bitlinear_status_string", l.status_string) ||
        !find(lib, "bitlinear_attention_workspace_size", l.attention_workspace_size) ||
        !find(lib, "bitlinear_attention", l.attention) || !find(lib, "bitlinear_cache_append", l.cache_append) ||
        !find(lib, "bitlinear_cache_read", l.cache_read) ||
        !find(lib, "bitlinear_attention_cached_workspace_size", l.attention_cached_workspace_size) ||
        !find(lib, "bitlinear_attention_cached", l.attention_cached) || !find(lib, "bitlinear_cache_evict", l.cache_evict) ||
        !find(lib, "bitlinear_rotate", l.rotate) ||
        !find(lib, "bitlinear_attention_shared_workspace_size", l.attention_shared_workspace_size) ||
        !find(lib, "bitlinear_attention_shared", l.attention_shared) || !find(lib, "bitlinear_cache_bounds", l.cache_bounds) ||
        !find(lib, "bitlinear_block_select_workspace_size", l.block_select_workspace_size) ||
        !find(lib, "bitlinear_block_select", l.block_select) ||
        !find(lib, "bitlinear_attention_selected_workspace_size", l.attention_selected_workspace_size) ||
        !find(lib, "bitlinear_attention_selected", l.attention_selected)) {
        PyErr_Format(error, "%s does not hold the attention calls: %s", path, lib ? "a symbol is missing" : dlerror());
        return nullptr;
    }
    g_lib = l;
    Py_INCREF(error);
    Py_XDECREF(g_error);
    g_error = error;
    Py_RETURN_NONE;
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr}, FAST(attention), FAST(cache_append), FAST(cache_read),
                         FAST(attention_cached), FAST(cache_evict), FAST(rotate), FAST(attention_shared), FAST(cache_bounds),
                         FAST(block_select), FAST(attention_selected), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
