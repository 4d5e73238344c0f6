// fastcall.cpp -- the way of the quantised-cache calls from Python to the C ABI
// when every argument is as it should be.
//
// Writing a decode step's tokens takes 2-3 us on the device; checking eight
// tensors in Python and passing fifteen arguments through ctypes takes 6 us
// on the host (measured: 9.3 us a call in all, 2.8 of them the launch).  The
// functions here make the same checks on the tensors themselves.  They never
// report an error: at the first argument that is not plainly right they return
// None, and the caller goes the long way, which makes the call or says what is
// wrong.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <indexcache.h>

namespace {

decltype(&ic_cache_write_q8) write_fn = nullptr;
decltype(&ic_cache_read_q8) read_fn = nullptr;
decltype(&ic_tree_attn_q8_paged) tree_fn = nullptr;

struct Declined {};
void need(bool ok) {
    if (!ok) throw Declined();
}

// A plain CUDA tensor on `device`.
const at::Tensor& tensor(PyObject* x, int64_t device) {
    need(THPVariable_CheckExact(x));
    const at::Tensor& t = THPVariable_Unpack(x);
    need(t.is_cuda() && t.get_device() == device && t.layout() == at::kStrided);
    return t;
}
void* dense(PyObject* x, at::ScalarType type, at::IntArrayRef shape, int64_t device) {
    const at::Tensor& t = tensor(x, device);
    need(t.scalar_type() == type && t.sizes() == shape && t.is_contiguous());
    return t.data_ptr();
}
void* rows_of(const at::Tensor& t, int64_t n, int64_t width, at::ScalarType type, int64_t& step) {
    need(t.dim() == 2 && t.size(0) == n && t.size(1) == width && t.scalar_type() == type);
    need(n == 0 || t.stride(1) == 1);
    step = n <= 1 ? width : t.stride(0);
    need(step >= width);
    return t.data_ptr();
}

PyObject* outcome(ic_status st) { return PyLong_FromLong((long)st); }

// (slots, ws, kv, kv_q8, kv_scale, k_idx, k_codes, k_scale, device, stream)
template <bool WRITE>
PyObject* cache_q8(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (n_args != 10) Py_RETURN_NONE;
    try {
        const int64_t device = PyLong_AsLongLong(a[8]);
        void* stream = PyLong_AsVoidPtr(a[9]);
        const bool latent = a[2] != Py_None, index = a[5] != Py_None;
        need(latent || index);
        need(latent == (a[3] != Py_None) && latent == (a[4] != Py_None));
        need(index == (a[6] != Py_None) && index == (a[7] != Py_None));
        const at::Tensor& rows = tensor(latent ? a[2] : a[5], device);
        const at::Tensor& cache = tensor(latent ? a[3] : a[6], device);
        need(rows.dim() == 2 && cache.dim() == 2);
        const int64_t n = rows.size(0), num_rows = cache.size(0);
        const at::ScalarType type = rows.scalar_type();
        need(type == at::kBFloat16 || type == at::kFloat);
        const ic_dtype dt = type == at::kFloat ? IC_F32 : IC_BF16;
        void *kv = nullptr, *kq = nullptr, *ks = nullptr, *ki = nullptr, *kc = nullptr, *sc = nullptr, *slots = nullptr;
        int64_t kv_step = 576, k_step = 128;
        if (latent) {
            kv = rows_of(rows, n, 576, type, kv_step);
            kq = dense(a[3], at::kByte, {num_rows, IC_Q8_ROW_BYTES}, device);
            ks = dense(a[4], at::kFloat, {num_rows}, device);
        }
        if (index) {
            ki = rows_of(tensor(a[5], device), n, 128, type, k_step);
            const at::ScalarType ct = tensor(a[6], device).scalar_type();
            need(ct == at::kByte || ct == at::kFloat8_e4m3fn);
            kc = dense(a[6], ct, {num_rows, 128}, device);
            sc = dense(a[7], at::kFloat, {num_rows}, device);
        }
        if (a[0] != Py_None) slots = dense(a[0], at::kInt, {n}, device);
        const at::Tensor& ws = tensor(a[1], device);
        const int64_t bytes = ws.numel();
        void* w = dense(a[1], at::kByte, {bytes}, device);
        ic_status st;
        Py_BEGIN_ALLOW_THREADS
        if (WRITE)
            st = write_fn(kv, kv_step, ki, k_step, dt, n, (const int32_t*)slots, kq, (float*)ks, kc, (float*)sc, num_rows, w,
                          (size_t)bytes, stream);
        else
            st = read_fn(kq, (const float*)ks, kc, (const float*)sc, num_rows, n, (const int32_t*)slots, dt, kv, kv_step, ki,
                         k_step, w, (size_t)bytes, stream);
        Py_END_ALLOW_THREADS
        return outcome(st);
    } catch (...) {
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

// (q, kv_q8, kv_scale, idx, tree, pr, scale, out, ws, device, stream)
PyObject* tree_attn_q8(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (n_args != 11) Py_RETURN_NONE;
    ic_paged_rows pr;
    {
        Py_buffer view;
        if (PyObject_GetBuffer(a[5], &view, PyBUF_SIMPLE) != 0) {
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        const bool fits = view.len == (Py_ssize_t)sizeof(pr);
        if (fits) memcpy(&pr, view.buf, sizeof(pr));
        PyBuffer_Release(&view);
        if (!fits) Py_RETURN_NONE;
    }
    try {
        const double scale = PyFloat_AsDouble(a[6]);
        need(!(scale == -1.0 && PyErr_Occurred()));
        const int64_t device = PyLong_AsLongLong(a[9]);
        void* stream = PyLong_AsVoidPtr(a[10]);
        const int64_t B = pr.B, Lq = pr.Lq, rows = (int64_t)pr.num_pages * pr.page_size;
        const at::Tensor& q = tensor(a[0], device);
        need(q.dim() == 4);
        const int64_t Hq = q.size(2);
        int64_t k = 0;
        void *idx = nullptr, *tree = nullptr;
        if (a[3] != Py_None) {
            const at::Tensor& t = tensor(a[3], device);
            need(t.dim() == 3 && t.size(2) > 0 && t.size(2) <= 16384);
            k = t.size(2);
            idx = dense(a[3], at::kInt, {B, Lq, k}, device);
        }
        if (a[4] != Py_None) tree = dense(a[4], at::kLong, {B, Lq}, device);
        void* pq = dense(a[0], at::kBFloat16, {B, Lq, Hq, 576}, device);
        void* kv = dense(a[1], at::kByte, {rows, IC_Q8_ROW_BYTES}, device);
        void* sc = dense(a[2], at::kFloat, {rows}, device);
        void* out = dense(a[7], at::kBFloat16, {B, Lq, Hq, 512}, device);
        const at::Tensor& ws = tensor(a[8], device);
        const int64_t bytes = ws.numel();
        void* w = dense(a[8], at::kByte, {bytes}, device);
        ic_status st;
        Py_BEGIN_ALLOW_THREADS
        st = tree_fn(pq, kv, (const float*)sc, (const int32_t*)idx, (int)k, (const uint64_t*)tree, &pr, (int)Hq, (float)scale,
                     out, w, (size_t)bytes, stream);
        Py_END_ALLOW_THREADS
        return outcome(st);
    } catch (...) {
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

// Addresses of ic_cache_write_q8, ic_cache_read_q8 and ic_tree_attn_q8_paged.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (n_args != 3) {
        PyErr_SetString(PyExc_TypeError, "bind: three addresses");
        return nullptr;
    }
    write_fn = reinterpret_cast<decltype(write_fn)>(PyLong_AsVoidPtr(a[0]));
    read_fn = reinterpret_cast<decltype(read_fn)>(PyLong_AsVoidPtr(a[1]));
    tree_fn = reinterpret_cast<decltype(tree_fn)>(PyLong_AsVoidPtr(a[2]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"cache_write_q8", FAST(&cache_q8<true>), nullptr},
                         {"cache_read_q8", FAST(&cache_q8<false>), nullptr},
                         {"tree_attn_q8", FAST(&tree_attn_q8), nullptr},
                         {"bind", FAST(&bind), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
