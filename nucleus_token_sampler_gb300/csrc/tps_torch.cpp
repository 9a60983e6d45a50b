// tps_torch.cpp -- the decode-step entry points on PyTorch tensors: argument checks, output tensors and the
// call of the C ABI, for decode.py.  A decode step's kernels take two to five microseconds, and the same
// work in Python takes ten to fifteen (attribute reads, two torch.empty, ctypes); here it takes two to three.
// The module knows nothing of the kernels: `bind` hands it the addresses of the library's entry points.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <optional>
#include <stdexcept>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/tps.h"

namespace {

decltype(&tps_qk_norm_rope) f_norm;
decltype(&tps_kv_write) f_write;
decltype(&tps_kv_read) f_read;
decltype(&tps_prefix_attention) f_attention;
bool bound;               // the pointers above are set
PyObject* on_error;       // called with (return code, entry point's name); raises
PyObject* out_of_memory;  // PyTorch's exception class

struct Raised {};  // a Python error is set

[[noreturn]] void refuse(const std::string& why) { throw std::invalid_argument(why); }

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// An output, from PyTorch's allocator without its operator dispatch (0.8 us less for each).
at::Tensor new_tensor(at::IntArrayRef shape, at::ScalarType type, c10::Device dev)
{
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

const char* type_name(at::ScalarType t) { return c10::toString(t); }

// A contiguous tensor of this type, shape and device.
void* dense(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, c10::Device dev)
{
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || t.sizes() != shape || t.device() != dev || !t.is_contiguous()) {
        std::string want = std::string(name) + " must be a contiguous " + type_name(type) + " tensor of shape (";
        for (size_t i = 0; i < shape.size(); ++i) want += (i ? ", " : "") + std::to_string(shape[i]);
        refuse(want + ") on " + dev.str());
    }
    return t.data_ptr();
}
void* dense_or_null(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, c10::Device dev)
{
    return o == Py_None ? nullptr : dense(o, name, shape, type, dev);
}

// A [T, heads, head_dim] CUDA tensor with head_dim contiguous, of `like`'s type and device if given.
const at::Tensor& heads(PyObject* o, const char* name, const at::Tensor* like)
{
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
        refuse(std::string(name) + " must be a CUDA tensor (there is no CPU path)");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.dim() != 3 || (t.stride(2) != 1 && t.size(2) > 1))
        refuse(std::string(name) + " must be [T, heads, head_dim] with unit stride along head_dim");
    if (like && (t.scalar_type() != like->scalar_type() || t.device() != like->device()))
        refuse(std::string(name) + " must be a " + type_name(like->scalar_type()) + " tensor on " + like->device().str());
    return t;
}

int dtype_code(at::ScalarType t)
{
    if (t == at::kBFloat16) return TPS_BF16;
    if (t == at::kFloat) return TPS_F32;
    throw c10::TypeError({__func__, __FILE__, __LINE__}, std::string("values must be float32 or bfloat16, got ") + type_name(t));
}

void check(int rc, const char* name)
{
    if (rc == TPS_OK) return;
    PyObject* r = PyObject_CallFunction(on_error, "is", rc, name);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
    throw Raised{};
}

void arity(Py_ssize_t have, Py_ssize_t want)
{
    if (have != want) refuse("wrong number of arguments");
}

int64_t whole(PyObject* o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

double number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}

bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v == 1;
}

// cache: (the bytes of a tps_kv_cache, device index)
const tps_kv_cache& cache_of(PyObject* bytes)
{
    if (!PyBytes_Check(bytes) || PyBytes_GET_SIZE(bytes) != (Py_ssize_t)sizeof(tps_kv_cache)) refuse("not a cache");
    return *reinterpret_cast<const tps_kv_cache*>(PyBytes_AS_STRING(bytes));
}

PyObject* pair(PyObject* a, PyObject* b)
{
    PyObject* r = PyTuple_New(2);
    if (!r) throw Raised{};
    PyTuple_SET_ITEM(r, 0, a);
    PyTuple_SET_ITEM(r, 1, b);
    return r;
}

PyObject* keep(PyObject* o)
{
    Py_INCREF(o);
    return o;
}

// q, k, q_weight, k_weight, positions, cos_sin, eps, interleaved, out, status
PyObject* norm(PyObject* const* a, Py_ssize_t n)
{
    arity(n, 10);
    const at::Tensor& q = heads(a[0], "q", nullptr);
    const at::Tensor& k = heads(a[1], "k", &q);
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hk = k.size(1);
    if (k.size(0) != T || k.size(2) != D) refuse("q and k must hold the same tokens and head size");
    const at::Tensor& cs = tensor(a[5], "cos_sin");
    if (cs.dim() != 2) refuse("cos_sin must be a float32 [positions, R] tensor");
    const int64_t R = cs.size(1);
    if (R % 2 || R > D) refuse("cos_sin must hold an even number of columns, at most the head size");
    const c10::Device dev = q.device();
    tps_norm_rope p = {};
    p.dtype = dtype_code(q.scalar_type());
    p.q = q.data_ptr();
    p.k = k.data_ptr();
    p.q_ld = q.stride(0), p.q_hd = q.stride(1), p.k_ld = k.stride(0), p.k_hd = k.stride(1);
    p.q_weight = static_cast<const float*>(dense_or_null(a[2], "q_weight", {D}, at::kFloat, dev));
    p.k_weight = static_cast<const float*>(dense_or_null(a[3], "k_weight", {D}, at::kFloat, dev));
    p.positions = static_cast<const int32_t*>(dense(a[4], "positions", {T}, at::kInt, dev));
    p.cos_sin = static_cast<const float*>(dense(a[5], "cos_sin", cs.sizes(), at::kFloat, dev));
    p.out_status = static_cast<int32_t*>(dense_or_null(a[9], "status", {T}, at::kInt, dev));
    p.T = T, p.n_positions = cs.size(0);
    if (Hq > INT32_MAX || Hk > INT32_MAX || D > INT32_MAX) refuse("too many heads or components");
    p.n_q_heads = (int32_t)Hq, p.n_k_heads = (int32_t)Hk, p.head_dim = (int32_t)D, p.rot_dim = (int32_t)R;
    p.eps = (float)number(a[6]);
    p.interleaved = truth(a[7]);
    const c10::cuda::CUDAGuard guard(dev);
    PyObject *oq, *ok;
    if (a[8] == Py_None) {
        at::Tensor x = new_tensor(q.sizes(), q.scalar_type(), dev), y = new_tensor(k.sizes(), k.scalar_type(), dev);
        p.out_q = x.data_ptr(), p.out_k = y.data_ptr();
        p.oq_ld = Hq * D, p.ok_ld = Hk * D, p.oq_hd = p.ok_hd = D;
        check(f_norm(&p, c10::cuda::getCurrentCUDAStream(dev.index()).stream()), "tps_qk_norm_rope");
        oq = THPVariable_Wrap(std::move(x)), ok = THPVariable_Wrap(std::move(y));
    } else {
        if (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 2) refuse("out must be a (q, k) pair");
        PyObject *px = PyTuple_GET_ITEM(a[8], 0), *py = PyTuple_GET_ITEM(a[8], 1);
        const at::Tensor& x = heads(px, "out[0]", &q);
        const at::Tensor& y = heads(py, "out[1]", &q);
        if (x.sizes() != q.sizes() || y.sizes() != k.sizes()) refuse("out must have the shapes of q and k");
        p.out_q = x.data_ptr(), p.out_k = y.data_ptr();
        p.oq_ld = x.stride(0), p.oq_hd = x.stride(1), p.ok_ld = y.stride(0), p.ok_hd = y.stride(1);
        check(f_norm(&p, c10::cuda::getCurrentCUDAStream(dev.index()).stream()), "tps_qk_norm_rope");
        oq = keep(px), ok = keep(py);
    }
    return pair(oq, ok);
}

// cache bytes, device index, k, v, slots
PyObject* write(PyObject* const* a, Py_ssize_t n)
{
    arity(n, 5);
    const tps_kv_cache& c = cache_of(a[0]);
    const at::Tensor& k = heads(a[2], "k", nullptr);
    const at::Tensor& v = heads(a[3], "v", &k);
    const int64_t T = k.size(0);
    const c10::Device dev(c10::kCUDA, (c10::DeviceIndex)whole(a[1]));
    if (k.size(1) != c.n_heads || k.size(2) != c.head_dim || v.sizes() != k.sizes() || k.device() != dev)
        refuse("k and v must be [T, " + std::to_string(c.n_heads) + ", " + std::to_string(c.head_dim) + "] on " + dev.str());
    const void* slots = dense(a[4], "slots", {T}, at::kLong, dev);
    const int code = dtype_code(k.scalar_type());
    const c10::cuda::CUDAGuard guard(dev);
    check(f_write(&c, k.data_ptr(), v.data_ptr(), code, T, k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                  static_cast<const int64_t*>(slots), c10::cuda::getCurrentCUDAStream(dev.index()).stream()),
          "tps_kv_write");
    return keep(Py_None);
}

// cache bytes, device index, slots, dtype code, out
PyObject* read(PyObject* const* a, Py_ssize_t n)
{
    arity(n, 5);
    const tps_kv_cache& c = cache_of(a[0]);
    const c10::Device dev(c10::kCUDA, (c10::DeviceIndex)whole(a[1]));
    const at::Tensor& s = tensor(a[2], "slots");
    if (s.dim() != 1) refuse("slots must be an int64 [T] tensor");
    const int64_t T = s.size(0);
    const int64_t* slots = static_cast<const int64_t*>(dense(a[2], "slots", {T}, at::kLong, dev));
    const int code = (int)whole(a[3]);
    const at::ScalarType type = code == TPS_BF16 ? at::kBFloat16 : at::kFloat;
    const int64_t shape[3] = {T, c.n_heads, c.head_dim};
    const c10::cuda::CUDAGuard guard(dev);
    void* stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    if (a[4] == Py_None) {
        at::Tensor k = new_tensor(shape, type, dev), v = new_tensor(shape, type, dev);
        check(f_read(&c, slots, T, k.data_ptr(), v.data_ptr(), code, stream), "tps_kv_read");
        PyObject* pk = THPVariable_Wrap(std::move(k));
        return pair(pk, THPVariable_Wrap(std::move(v)));
    }
    if (!PyTuple_Check(a[4]) || PyTuple_GET_SIZE(a[4]) != 2) refuse("out must be a (k, v) pair");
    PyObject *pk = PyTuple_GET_ITEM(a[4], 0), *pv = PyTuple_GET_ITEM(a[4], 1);
    void *ok = dense(pk, "out[0]", shape, type, dev), *ov = dense(pv, "out[1]", shape, type, dev);
    check(f_read(&c, slots, T, ok, ov, code, stream), "tps_kv_read");
    return pair(keep(pk), keep(pv));
}

// q, cache bytes, device index, prefix_pages, prefix_len, page_table, suffix_len, scale (None: D ** -0.5), want_lse, out, status, workspace
PyObject* attention(PyObject* const* a, Py_ssize_t n)
{
    arity(n, 12);
    if (!THPVariable_Check(a[0])) refuse("q must be a tensor");
    const at::Tensor& q = THPVariable_Unpack(a[0]);
    if (!q.is_cuda() || q.scalar_type() != at::kBFloat16 || (q.dim() != 3 && q.dim() != 4) || !q.is_contiguous())
        refuse("q must be a contiguous bfloat16 CUDA tensor [B, heads, D] or [B, tokens, heads, D]");
    const tps_kv_cache& c = cache_of(a[1]);
    const c10::Device dev(c10::kCUDA, (c10::DeviceIndex)whole(a[2]));
    const int64_t B = q.size(0), Hq = q.size(-2), D = q.size(-1);
    if (q.device() != dev || D != c.head_dim) refuse("q must have head size " + std::to_string(c.head_dim) + " and be on " + dev.str());
    if (D != 64 && D != 128) refuse("prefix_attention takes head sizes 64 and 128");
    if (Hq % c.n_heads || Hq > INT32_MAX) refuse("the query heads must be a multiple of the cache's " + std::to_string(c.n_heads) + " heads");
    const at::Tensor& pages = tensor(a[3], "prefix_pages");
    const int64_t prefix = whole(a[4]);
    if (pages.dim() != 1 || prefix < 0 || pages.size(0) * c.page_size < prefix)
        refuse("prefix_pages must be an int32 [n] tensor whose pages hold prefix_len tokens");
    const at::Tensor& table = tensor(a[5], "page_table");
    if (table.dim() != 2 || table.size(0) != B || table.scalar_type() != at::kInt || table.device() != dev ||
        (table.size(1) > 1 && table.stride(1) != 1))
        refuse("page_table must be an int32 [" + std::to_string(B) + ", W] tensor with unit stride along W on " + dev.str());
    tps_attention p = {};
    p.q = q.data_ptr();
    p.prefix_pages = static_cast<const int32_t*>(dense(a[3], "prefix_pages", pages.sizes(), at::kInt, dev));
    p.page_table = static_cast<const int32_t*>(table.data_ptr());
    p.suffix_len = static_cast<const int32_t*>(dense(a[6], "suffix_len", {B}, at::kInt, dev));
    p.out_status = static_cast<int32_t*>(dense_or_null(a[10], "status", {B}, at::kInt, dev));
    if (a[11] != Py_None) {
        const at::Tensor& w = tensor(a[11], "workspace");
        if (w.device() != dev || !w.is_contiguous()) refuse("workspace must be a contiguous tensor on " + dev.str());
        p.workspace = w.data_ptr();
        p.workspace_bytes = (int64_t)w.nbytes();
    }
    p.B = B, p.prefix_len = prefix, p.table_width = table.size(1), p.table_ld = B > 1 ? table.stride(0) : table.size(1);
    const int64_t tokens = q.dim() == 4 ? q.size(1) : 1;
    if (tokens > INT32_MAX) refuse("too many query tokens");
    p.q_len = (int32_t)tokens, p.n_q_heads = (int32_t)Hq;
    p.scale = a[7] == Py_None ? (D == 64 ? 0.125f : 0.08838834764831845f) : (float)number(a[7]);
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor out, lse;
    if (a[9] == Py_None) {
        out = new_tensor(q.sizes(), at::kBFloat16, dev);
        p.out = out.data_ptr();
    } else {
        p.out = dense(a[9], "out", q.sizes(), at::kBFloat16, dev);
    }
    const bool want = truth(a[8]);
    if (want) {
        lse = new_tensor(q.sizes().slice(0, q.dim() - 1), at::kFloat, dev);
        p.out_lse = static_cast<float*>(lse.data_ptr());
    }
    check(f_attention(&c, &p, c10::cuda::getCurrentCUDAStream(dev.index()).stream()), "tps_prefix_attention");
    PyObject* r = a[9] == Py_None ? THPVariable_Wrap(std::move(out)) : keep(a[9]);
    return want ? pair(r, THPVariable_Wrap(std::move(lse))) : r;
}

PyObject* bind(PyObject* const* a, Py_ssize_t n)
{
    arity(n, 6);
    auto address = [](PyObject* o) { return reinterpret_cast<void*>(PyLong_AsVoidPtr(o)); };
    f_norm = reinterpret_cast<decltype(f_norm)>(address(a[0]));
    f_write = reinterpret_cast<decltype(f_write)>(address(a[1]));
    f_read = reinterpret_cast<decltype(f_read)>(address(a[2]));
    f_attention = reinterpret_cast<decltype(f_attention)>(address(a[3]));
    Py_INCREF(a[4]);
    Py_XSETREF(on_error, a[4]);
    Py_INCREF(a[5]);
    Py_XSETREF(out_of_memory, a[5]);
    bound = f_norm && f_write && f_read && f_attention;
    return keep(Py_None);
}

// C++ exceptions become Python ones here; none leaves the module.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    try {
        if (!bound && F != bind) throw std::runtime_error("the module is not bound to the library");
        return F(a, n);
    } catch (const Raised&) {
        return nullptr;
    } catch (const c10::TypeError& e) {
        PyErr_SetString(PyExc_TypeError, e.what_without_backtrace());
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(out_of_memory ? out_of_memory : PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define TPS_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TPS_METHOD(bind), TPS_METHOD(norm), TPS_METHOD(write), TPS_METHOD(read), TPS_METHOD(attention),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tps_torch", "The decode-step entry points on tensors.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__tps_torch() { return PyModule_Create(&module); }
