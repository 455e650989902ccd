// marshal.cpp -- argument marshalling for the entry points over heads: checks
// the tensors a Python caller passes, allocates its results, fills the C
// argument structs and calls the library.  A Python extension module, because
// these calls take a dozen tensors each and run for a few microseconds: checked
// attribute by attribute in Python, the arguments would cost more than the
// kernels.  The library's functions are handed over by address (bind), so the
// module uses whichever build of it the Python side has opened.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <cmath>
#include <initializer_list>
#include <optional>

#include "rdx.h"

namespace {

template <class Args>
using Entry = rdx_status (*)(const Args*, cudaStream_t);

struct Library {
    Entry<rdx_qk_norm_rope_args> norm = nullptr;
    Entry<rdx_qk_norm_rope_grad_args> norm_grad = nullptr;
    size_t (*norm_grad_workspace)(int) = nullptr;
    Entry<rdx_kv_rows_args> write = nullptr;
    Entry<rdx_kv_rows_args> read = nullptr;
    Entry<rdx_kv_attend_args> attend = nullptr;
    size_t (*attend_workspace)(const rdx_kv_attend_args*) = nullptr;
    PyObject* cache_type = nullptr;  // abi.KVCache
    PyObject* fail = nullptr;        // raises abi.RdxError(name, status)
} g_lib;
PyObject* g_tensors = nullptr;       // attribute names
PyObject* g_cuda_stream = nullptr;

// The call in hand: its name for messages, device, stream and the guards that
// make both current while results are allocated and kernels launched.
struct Call {
    const char* name;
    int device;
    cudaStream_t stream;
    std::optional<c10::cuda::CUDAGuard> on_device;
    std::optional<c10::cuda::CUDAStreamGuard> on_stream;

    Call(const char* n, int dev, PyObject* given) : name(n), device(dev) {
        if (given == nullptr || given == Py_None) {
            if (c10::cuda::current_device() != dev) on_device.emplace(c10::DeviceIndex(dev));
            stream = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream();
            return;
        }
        PyObject* handle = PyObject_GetAttr(given, g_cuda_stream);
        if (handle == nullptr) throw python_error();
        stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(handle));
        Py_DECREF(handle);
        if (PyErr_Occurred()) throw python_error();
        on_stream.emplace(c10::cuda::getStreamFromExternal(stream, c10::DeviceIndex(dev)));
    }
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
        return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, c10::DeviceIndex(device)), std::nullopt);
    }
};

bool absent(PyObject* o) { return o == nullptr || o == Py_None; }

const at::Tensor& tensor(const char* name, const char* what, PyObject* o) {
    TORCH_CHECK_TYPE(o != nullptr && THPVariable_Check(o), name, ": ", what, " must be a tensor");
    return THPVariable_Unpack(o);
}

// The first argument decides device and type.
const at::Tensor& leading(const char* name, const char* what, PyObject* o) {
    const at::Tensor& x = tensor(name, what, o);
    TORCH_CHECK_TYPE(x.is_cuda(), name, ": ", what, " must be a CUDA tensor");
    TORCH_CHECK_TYPE(x.scalar_type() == at::kFloat || x.scalar_type() == at::kBFloat16, name, ": ", what,
                     " must be float32 or bfloat16, got ", x.scalar_type());
    TORCH_CHECK_TYPE(x.dim() == 3, name, ": ", what, " must have 3 dimensions, got ", x.dim());
    return x;
}
int type_code(const at::Tensor& x) { return x.scalar_type() == at::kFloat ? RDX_TYPE_F32 : RDX_TYPE_BF16; }

void check_kind(const Call& c, const char* what, const at::Tensor& x, at::ScalarType type) {
    TORCH_CHECK_TYPE(x.is_cuda() && x.get_device() == c.device && x.scalar_type() == type, c.name, ": ", what, " must be a ",
                     type, " tensor on CUDA device ", c.device);
}
// [tokens, heads, head_dim] rows; `shape` empty: any.
rdx_heads rows(const Call& c, const char* what, const at::Tensor& x, at::ScalarType type, at::IntArrayRef shape) {
    check_kind(c, what, x, type);
    TORCH_CHECK_TYPE(x.dim() == 3, c.name, ": ", what, " must have 3 dimensions, got ", x.dim());
    TORCH_CHECK_VALUE(shape.empty() || x.sizes() == shape, c.name, ": ", what, " must have shape ", shape, ", got ", x.sizes());
    TORCH_CHECK_VALUE(x.stride(2) == 1 || x.size(2) <= 1, c.name, ": the last dimension of ", what, " must be contiguous");
    return {x.data_ptr(), x.stride(0), x.stride(1)};
}
// A contiguous tensor of one shape.
template <class T>
T* plain(const Call& c, const char* what, PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor& x = tensor(c.name, what, o);
    check_kind(c, what, x, type);
    TORCH_CHECK_VALUE(x.sizes() == shape && x.is_contiguous(), c.name, ": ", what, " must be contiguous with shape ", shape,
                      ", got ", x.sizes());
    return static_cast<T*>(x.data_ptr());
}
// A result: the caller's, or a new tensor.
at::Tensor result(const Call& c, const char* what, PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
    return absent(o) ? c.empty(shape, type) : tensor(c.name, what, o);
}
at::Tensor workspace(const Call& c, PyObject* o, size_t need) {
    if (absent(o)) return c.empty({int64_t(need)}, at::kByte);
    const at::Tensor& x = tensor(c.name, "workspace", o);
    TORCH_CHECK_VALUE(x.is_cuda() && x.get_device() == c.device && x.is_contiguous(), c.name,
                      ": workspace must be a contiguous tensor on CUDA device ", c.device);
    return x;
}

// One of a cache's four tensors, as it is now: a caller may have moved its
// storage, or given it back, since the cache was made.
char* cache_part(const char* name, const char* what, const at::Tensor& x, at::ScalarType type, int device, at::IntArrayRef shape) {
    TORCH_CHECK_TYPE(x.is_cuda() && x.get_device() == device && x.scalar_type() == type, name, ": the KVCache's ", what,
                     " must be a ", type, " tensor on CUDA device ", device);
    TORCH_CHECK_VALUE(x.sizes() == shape && x.is_contiguous(), name, ": the KVCache's ", what,
                      " must be contiguous with shape ", shape, ", got ", x.sizes());
    const size_t need = x.numel() == 0 ? 0 : size_t(x.storage_offset() + x.numel()) * x.element_size();
    TORCH_CHECK_VALUE(x.storage().nbytes() >= need, name, ": the memory of the KVCache's ", what, " is gone");
    return static_cast<char*>(x.data_ptr());
}
struct CacheTensors {
    THPObjectPtr held;  // the tuple of them
    const at::Tensor& operator[](int i) const { return THPVariable_Unpack(PyTuple_GET_ITEM(held.get(), i)); }
};
rdx_kv_cache cache_of(const char* name, PyObject* o, int* device, CacheTensors& x) {
    TORCH_CHECK_TYPE(o != nullptr && PyObject_TypeCheck(o, reinterpret_cast<PyTypeObject*>(g_lib.cache_type)), name,
                     ": cache must be a KVCache");
    x.held = PyObject_GetAttr(o, g_tensors);
    PyObject* const parts = x.held.get();
    if (parts == nullptr) throw python_error();
    bool fits = PyTuple_Check(parts) && PyTuple_GET_SIZE(parts) == 4;
    for (int i = 0; fits && i < 4; ++i) fits = THPVariable_Check(PyTuple_GET_ITEM(parts, i));
    TORCH_CHECK_TYPE(fits, name, ": not a KVCache of this library");
    const at::Tensor& k = x[0];
    const at::ScalarType type = k.scalar_type();
    TORCH_CHECK_TYPE(k.is_cuda() && k.dim() == 4 && (type == at::kChar || type == at::kFloat8_e4m3fn), name,
                     ": the KVCache's k must be a 4-D CUDA tensor of 8-bit codes");
    const at::IntArrayRef shape = k.sizes();
    for (int i = 1; i < 4; ++i)
        TORCH_CHECK_VALUE(shape[i] >= 1 && shape[i] <= INT32_MAX, name, ": a KVCache of shape ", shape);
    *device = k.get_device();
    rdx_kv_cache c = {};
    c.k = cache_part(name, "k", k, type, *device, shape);
    c.v = cache_part(name, "v", x[1], type, *device, shape);
    c.k_scale = reinterpret_cast<float*>(cache_part(name, "k_scale", x[2], at::kFloat, *device, shape.slice(0, 3)));
    c.v_scale = reinterpret_cast<float*>(cache_part(name, "v_scale", x[3], at::kFloat, *device, shape.slice(0, 3)));
    c.pages = shape[0];
    c.heads = int32_t(shape[1]);
    c.page_size = int32_t(shape[2]);
    c.head_dim = int32_t(shape[3]);
    c.format = type == at::kChar ? RDX_KV_INT8 : RDX_KV_E4M3;
    return c;
}

// The call writes into this tensor of the caller's: operations that saved it
// for their gradients are told.
void written(const at::Tensor& x) {
    if (!x.is_inference()) x.unsafeGetTensorImpl()->bump_version();
}
void written(PyObject* o) {
    if (!absent(o)) written(THPVariable_Unpack(o));
}

template <class Args>
bool launched(const Call& c, Entry<Args> entry, const Args& args) {
    rdx_status st;
    Py_BEGIN_ALLOW_THREADS  // a launch waits where the queue before it is full
    st = entry(&args, c.stream);
    Py_END_ALLOW_THREADS
    if (st == RDX_OK) return true;
    PyObject* r = PyObject_CallFunction(g_lib.fail, "si", c.name, int(st));
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, c.name);
    return false;
}

double number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
}
bool truth(PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw python_error();
    return x != 0;
}
PyObject* wrapped(const at::Tensor& a, const at::Tensor& b) {
    PyObject *x = THPVariable_Wrap(a), *y = THPVariable_Wrap(b);
    PyObject* t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

// Fields that the norm and its gradient share.  args: q, k, q_weight, k_weight,
// positions, cos, sin, eps, interleaved; y: the output or the incoming gradient.
rdx_qk_norm_rope_args norm_args(const Call& c, PyObject* const* args, const at::Tensor& q, const at::Tensor& k,
                                const char* q_what, const at::Tensor& qy, const char* k_what, const at::Tensor& ky) {
    const at::ScalarType type = q.scalar_type();
    const int64_t tokens = q.size(0), dim = q.size(2);
    TORCH_CHECK_VALUE(k.size(0) == tokens && k.size(2) == dim, c.name, ": q ", q.sizes(), " and k ", k.sizes(),
                      " differ in tokens or head_dim");
    TORCH_CHECK_VALUE(dim <= INT32_MAX && q.size(1) <= INT32_MAX && k.size(1) <= INT32_MAX, c.name, ": too many heads or values");
    rdx_qk_norm_rope_args a = {};
    a.q = rows(c, "q", q, type, {});
    a.k = rows(c, "k", k, type, {});
    a.q_out = rows(c, q_what, qy, type, q.sizes());
    a.k_out = rows(c, k_what, ky, type, k.sizes());
    a.q_weight = plain<float>(c, "q_weight", args[2], at::kFloat, {dim});
    a.k_weight = plain<float>(c, "k_weight", args[3], at::kFloat, {dim});
    if (!absent(args[5])) {
        const at::Tensor& cos = tensor(c.name, "cos", args[5]);
        TORCH_CHECK_VALUE(cos.dim() == 2 && cos.size(1) <= INT32_MAX / 2, c.name, ": cos must be [positions, rot_dim / 2]");
        a.positions = plain<int64_t>(c, "positions", args[4], at::kLong, {tokens});
        a.cos = plain<float>(c, "cos", args[5], at::kFloat, cos.sizes());
        a.sin = plain<float>(c, "sin", args[6], at::kFloat, cos.sizes());
        a.max_pos = cos.size(0);
        a.rot_dim = int32_t(2 * cos.size(1));
    }
    a.tokens = tokens;
    a.q_heads = int32_t(q.size(1));
    a.k_heads = int32_t(k.size(1));
    a.head_dim = int32_t(dim);
    a.interleaved = truth(args[8]);
    a.type = type_code(q);
    a.eps = float(number(args[7]));
    return a;
}

// Whether autograd follows any of these (None and what is no tensor: not).
bool followed(std::initializer_list<PyObject*> tensors) {
    if (!at::GradMode::is_enabled()) return false;
    for (PyObject* o : tensors)
        if (o != nullptr && THPVariable_Check(o) && THPVariable_Unpack(o).requires_grad()) return true;
    return false;
}

// NotImplemented where autograd follows an argument: abi.py has the function
// that it calls back.
PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const char* name = "rdx_qk_norm_rope";
    const at::Tensor& q = leading(name, "q", args[0]);
    const at::Tensor& k = leading(name, "k", args[1]);
    if (followed({args[0], args[1], args[2], args[3], args[5], args[6], args[9], args[10]})) {
        Py_INCREF(Py_NotImplemented);
        return Py_NotImplemented;
    }
    const Call c(name, q.get_device(), args[11]);
    const at::Tensor qo = result(c, "q_out", args[9], q.scalar_type(), q.sizes());
    const at::Tensor ko = result(c, "k_out", args[10], q.scalar_type(), k.sizes());
    const rdx_qk_norm_rope_args a = norm_args(c, args, q, k, "q_out", qo, "k_out", ko);
    if (!launched(c, g_lib.norm, a)) return nullptr;
    written(args[9]);
    written(args[10]);
    return wrapped(qo, ko);
    END_HANDLE_TH_ERRORS
}

// args: as norm_args, then dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace, stream
PyObject* qk_norm_rope_grad(PyObject*, PyObject* const* args, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const char* name = "rdx_qk_norm_rope_grad";
    const at::Tensor& q = leading(name, "q", args[0]);
    const at::Tensor& k = leading(name, "k", args[1]);
    const Call c(name, q.get_device(), args[16]);
    const at::ScalarType type = q.scalar_type();
    rdx_qk_norm_rope_grad_args a = {};
    a.fwd = norm_args(c, args, q, k, "dq_out", tensor(name, "dq_out", args[9]), "dk_out", tensor(name, "dk_out", args[10]));
    const at::Tensor dq = result(c, "dq", args[11], type, q.sizes()), dk = result(c, "dk", args[12], type, k.sizes());
    at::Tensor dw[2];
    for (int i = 0; i < 2; ++i) dw[i] = result(c, "weight gradient", args[13 + i], at::kFloat, {q.size(2)});
    for (const at::Tensor& w : dw) {
        check_kind(c, "weight gradient", w, at::kFloat);
        TORCH_CHECK_VALUE(w.dim() == 1 && w.size(0) == q.size(2) && w.is_contiguous(), name,
                          ": a weight gradient must be contiguous with shape [", q.size(2), "]");
    }
    const at::Tensor ws = workspace(c, args[15], g_lib.norm_grad_workspace(int(q.size(2))));
    a.dq = rows(c, "dq", dq, type, q.sizes());
    a.dk = rows(c, "dk", dk, type, k.sizes());
    a.dq_weight = static_cast<float*>(dw[0].data_ptr());
    a.dk_weight = static_cast<float*>(dw[1].data_ptr());
    a.workspace = ws.data_ptr();
    a.workspace_bytes = ws.nbytes();
    if (!launched(c, g_lib.norm_grad, a)) return nullptr;
    for (int i = 11; i < 15; ++i) written(args[i]);
    PyObject* out[4] = {THPVariable_Wrap(dq), THPVariable_Wrap(dk), THPVariable_Wrap(dw[0]), THPVariable_Wrap(dw[1])};
    PyObject* t = out[0] && out[1] && out[2] && out[3] ? PyTuple_Pack(4, out[0], out[1], out[2], out[3]) : nullptr;
    for (PyObject* o : out) Py_XDECREF(o);
    return t;
    END_HANDLE_TH_ERRORS
}

// args: cache, k, v, slots, stream
PyObject* kv_write(PyObject*, PyObject* const* args, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const char* name = "rdx_kv_write";
    int device = 0;
    rdx_kv_rows_args a = {};
    CacheTensors cache;
    a.cache = cache_of(name, args[0], &device, cache);
    const at::Tensor& k = leading(name, "k", args[1]);
    const Call c(name, device, args[4]);
    const int64_t shape[3] = {k.size(0), a.cache.heads, a.cache.head_dim};
    a.k = rows(c, "k", k, k.scalar_type(), shape);
    a.v = rows(c, "v", tensor(name, "v", args[2]), k.scalar_type(), shape);
    a.slots = plain<int64_t>(c, "slots", args[3], at::kLong, {shape[0]});
    a.tokens = shape[0];
    a.type = type_code(k);
    if (!launched(c, g_lib.write, a)) return nullptr;
    for (int i = 0; i < 4; ++i) written(cache[i]);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// args: cache, slots, type code, k_out, v_out, stream
PyObject* kv_read(PyObject*, PyObject* const* args, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const char* name = "rdx_kv_read";
    int device = 0;
    rdx_kv_rows_args a = {};
    CacheTensors cache;
    a.cache = cache_of(name, args[0], &device, cache);
    const Call c(name, device, args[5]);
    const at::Tensor& slots = tensor(name, "slots", args[1]);
    TORCH_CHECK_VALUE(slots.dim() == 1, name, ": slots must have one dimension");
    const int64_t shape[3] = {slots.size(0), a.cache.heads, a.cache.head_dim};
    const at::ScalarType type = PyLong_AsLong(args[2]) == RDX_TYPE_F32 ? at::kFloat : at::kBFloat16;
    const at::Tensor k = result(c, "k_out", args[3], type, shape), v = result(c, "v_out", args[4], type, shape);
    a.k = rows(c, "k_out", k, type, shape);
    a.v = rows(c, "v_out", v, type, shape);
    a.slots = plain<int64_t>(c, "slots", args[1], at::kLong, {shape[0]});
    a.tokens = shape[0];
    a.type = type_code(k);
    if (!launched(c, g_lib.read, a)) return nullptr;
    written(args[3]);
    written(args[4]);
    return wrapped(k, v);
    END_HANDLE_TH_ERRORS
}

// args: q, cache, block_table, lens, scale, max_len, out, lse, workspace, stream
PyObject* kv_attend(PyObject*, PyObject* const* args, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const char* name = "rdx_kv_attend";
    int device = 0;
    const at::Tensor& q = leading(name, "q", args[0]);
    rdx_kv_attend_args a = {};
    CacheTensors cache;
    a.cache = cache_of(name, args[1], &device, cache);
    const Call c(name, device, args[9]);
    const int64_t batch = q.size(0), heads = q.size(1), dim = q.size(2);
    TORCH_CHECK_VALUE(dim == a.cache.head_dim, name, ": q has head_dim ", dim, ", the cache ", a.cache.head_dim);
    TORCH_CHECK_VALUE(heads <= INT32_MAX, name, ": too many heads");
    const at::Tensor& table = tensor(name, "block_table", args[2]);
    check_kind(c, "block_table", table, at::kInt);
    TORCH_CHECK_VALUE(table.dim() == 2 && table.size(0) == batch, name, ": block_table must be [", batch, ", pages]");
    TORCH_CHECK_VALUE(table.size(1) <= 1 || table.stride(1) == 1, name, ": the rows of block_table must be contiguous");
    const at::Tensor out = result(c, "out", args[6], q.scalar_type(), q.sizes());
    a.q = rows(c, "q", q, q.scalar_type(), {});
    a.out = rows(c, "out", out, q.scalar_type(), q.sizes());
    a.block_table = static_cast<const int32_t*>(table.data_ptr());
    a.lens = plain<int32_t>(c, "lens", args[3], at::kInt, {batch});
    if (!absent(args[7])) a.lse = plain<float>(c, "lse", args[7], at::kFloat, {batch, heads});
    a.batch = batch;
    a.table_stride = table.stride(0);
    a.table_pages = table.size(1);
    const int64_t all = table.size(1) > INT32_MAX / a.cache.page_size ? INT32_MAX : table.size(1) * a.cache.page_size;
    a.max_len = absent(args[5]) ? all : PyLong_AsLongLong(args[5]);
    if (PyErr_Occurred()) throw python_error();
    a.q_heads = int32_t(heads);
    a.type = type_code(q);
    a.scale = float(absent(args[4]) ? 1.0 / std::sqrt(double(dim)) : number(args[4]));
    const size_t need = g_lib.attend_workspace(&a);
    at::Tensor ws;
    if (need > 0) {
        ws = workspace(c, args[8], need);
        a.workspace = ws.data_ptr();
        a.workspace_bytes = ws.nbytes();
    }
    if (!launched(c, g_lib.attend, a)) return nullptr;
    written(args[6]);
    written(args[7]);
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// args: the library functions' addresses in the order of Library, the KVCache
// type, the function that raises RdxError
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 9) {
        PyErr_SetString(PyExc_TypeError, "bind takes 9 arguments");
        return nullptr;
    }
    void* at[7];
    for (int i = 0; i < 7; ++i) {
        at[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    if (!PyType_Check(args[7]) || !PyCallable_Check(args[8])) {
        PyErr_SetString(PyExc_TypeError, "bind takes a type and a function at the end");
        return nullptr;
    }
    g_lib.norm = reinterpret_cast<Entry<rdx_qk_norm_rope_args>>(at[0]);
    g_lib.norm_grad = reinterpret_cast<Entry<rdx_qk_norm_rope_grad_args>>(at[1]);
    g_lib.norm_grad_workspace = reinterpret_cast<size_t (*)(int)>(at[2]);
    g_lib.write = reinterpret_cast<Entry<rdx_kv_rows_args>>(at[3]);
    g_lib.read = reinterpret_cast<Entry<rdx_kv_rows_args>>(at[4]);
    g_lib.attend = reinterpret_cast<Entry<rdx_kv_attend_args>>(at[5]);
    g_lib.attend_workspace = reinterpret_cast<size_t (*)(const rdx_kv_attend_args*)>(at[6]);
    Py_INCREF(args[7]);
    Py_INCREF(args[8]);
    g_lib.cache_type = args[7];
    g_lib.fail = args[8];
    Py_RETURN_NONE;
}

// Each function takes exactly its arguments, by position: abi.py has the
// signatures, defaults and documentation.
template <PyObject* (*kFn)(PyObject*, PyObject* const*, Py_ssize_t), int kArgs>
PyObject* counted(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    if (n != kArgs || g_lib.fail == nullptr) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments after bind, got %zd", kArgs, n);
        return nullptr;
    }
    return kFn(self, args, n);
}
template <PyObject* (*kFn)(PyObject*, PyObject* const*, Py_ssize_t), int kArgs>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&counted<kFn, kArgs>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
    method<qk_norm_rope, 12>("qk_norm_rope"),
    method<qk_norm_rope_grad, 17>("qk_norm_rope_grad"),
    method<kv_write, 5>("kv_write"),
    method<kv_read, 6>("kv_read"),
    method<kv_attend, 10>("kv_attend"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
    g_tensors = PyUnicode_InternFromString("_tensors");
    g_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    PyObject* m = g_tensors && g_cuda_stream ? PyModule_Create(&g_module) : nullptr;
    // abi.py compares it: the module reads tensors through this version's headers
    if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", RDX_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
