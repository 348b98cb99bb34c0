// binding_native.cpp -- the paged calls of binding.py with their arguments
// marshalled in C++.  A serving step makes several of them in the time that
// their kernels take, and a call through Python checks and ctypes is 15 to 19 us
// of host time, of which the launches are 2.5 to 5.
//
// Each function takes the call's arguments in order and serves the regular
// case: plain contiguous CUDA tensors of the expected types and ranks on the
// current device, outputs and workspace to be allocated.  For anything else, and
// where the C ABI refuses, it does nothing and returns None: binding.py then
// makes the call the long way, and raises what there is to raise.
#include <Python.h>
#include <dlfcn.h>

#include <initializer_list>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "csa.h"

namespace {

// the C ABI, from the library that binding.py loaded (bind)
struct Abi {
    decltype(&::csa_plan_workspace_bytes) plan_bytes;
    decltype(&::csa_plan_pages) plan;
    decltype(&::csa_paged_write) write;
    decltype(&::csa_paged_write_fp8kv) write_fp8;
    decltype(&::csa_attend_paged_workspace_bytes) attend_bytes;
    decltype(&::hca_attend_paged) attend;
    decltype(&::hca_attend_paged_fp8kv) attend_fp8;
} abi;

// Arguments as they are read; `ok` turns false at the first that is not regular.
struct Args {
    PyObject *const *at;
    Py_ssize_t n;
    int device = -1;
    bool ok;

    Args(PyObject *const *args, Py_ssize_t have, Py_ssize_t want) : at(args), n(have), ok(have == want && abi.plan) {}

    // argument i: a contiguous tensor of `dims` dimensions (-1: any), on the device of the first one
    const at::Tensor *tensor(Py_ssize_t i, at::ScalarType type, int dims) {
        return of(ok ? at[i] : nullptr, type, dims);
    }
    const at::Tensor *optional(Py_ssize_t i, at::ScalarType type, int dims) {
        return !ok || at[i] == Py_None ? nullptr : of(at[i], type, dims);
    }
    const at::Tensor *of(PyObject *o, at::ScalarType type, int dims) {
        if (!ok || !THPVariable_CheckExact(o)) return fail();
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.scalar_type() != type || t.layout() != at::kStrided || (dims >= 0 && t.dim() != dims) ||
            !t.is_contiguous())
            return fail();
        if (device < 0 && (device = t.get_device()) != c10::cuda::current_device()) return fail();
        return t.get_device() == device ? &t : fail();
    }
    long long integer(Py_ssize_t i, long long most = 0x7fffffffLL) {
        if (!ok || !PyLong_CheckExact(at[i])) return fail(), 0;
        int over = 0;
        const long long v = PyLong_AsLongLongAndOverflow(at[i], &over);
        if (over || v < -most || v > most) fail();
        return v;
    }
    double real(Py_ssize_t i) {
        if (ok && PyFloat_CheckExact(at[i])) return PyFloat_AS_DOUBLE(at[i]);
        return (double)integer(i);
    }
    const at::Tensor *fail() {
        ok = false;
        return nullptr;
    }
};

template <typename T>
const T *ptr(const at::Tensor *t) {
    return t ? static_cast<const T *>(t->data_ptr()) : nullptr;
}

void *stream_of(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

at::Tensor bytes_like(const at::Tensor &t, size_t n) {
    return n ? at::empty({(int64_t)n}, t.options().dtype(at::kByte)) : at::Tensor();
}

template <typename F>
int call(F f) {  // without the interpreter's lock
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
    return rc;
}

// n elements of buf's storage from byte `at` on, as a tensor of its own
at::Tensor part(const at::Tensor &buf, at::ScalarType type, int64_t at, int64_t n) {
    const caffe2::TypeMeta meta = c10::scalarTypeToTypeMeta(type);
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buf.storage()), buf.key_set(), meta);
    t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    t.unsafeGetTensorImpl()->set_storage_offset(at / (int64_t)meta.itemsize());
    return t;
}

PyObject *bind(PyObject *, PyObject *path) {
    const char *name = PyUnicode_AsUTF8(path);
    if (!name) return nullptr;
    void *lib = dlopen(name, RTLD_NOW);
    Abi a = {};
    const auto find = [&](auto &f, const char *symbol) {
        f = reinterpret_cast<std::decay_t<decltype(f)>>(lib ? dlsym(lib, symbol) : nullptr);
        return f != nullptr;
    };
    if (!find(a.plan_bytes, "csa_plan_workspace_bytes") || !find(a.plan, "csa_plan_pages") ||
        !find(a.write, "csa_paged_write") || !find(a.write_fp8, "csa_paged_write_fp8kv") ||
        !find(a.attend_bytes, "csa_attend_paged_workspace_bytes") || !find(a.attend, "hca_attend_paged") ||
        !find(a.attend_fp8, "hca_attend_paged_fp8kv"))
        return PyErr_Format(PyExc_RuntimeError, "%s lacks the paged calls", name);
    abi = a;
    Py_RETURN_NONE;
}

// old_len, new_len, free_pages, block_table, m, page, ring_rows, max_tokens, max_entries
PyObject *plan_pages(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 9);
    const at::Tensor *old_len = a.tensor(0, at::kInt, 1), *new_len = a.tensor(1, at::kInt, 1),
                     *free_pages = a.tensor(2, at::kInt, 1), *table = a.tensor(3, at::kInt, 2);
    const long long m = a.integer(4), page = a.integer(5), ring = a.integer(6), tokens = a.integer(7), entries = a.integer(8);
    if (!a.ok || tokens < 0 || entries < 0) Py_RETURN_NONE;
    const int64_t batch = table->size(0), columns = table->size(1);
    if (old_len->size(0) != batch || new_len->size(0) != batch || batch > (1 << 20) || columns > 0x7fffffff) Py_RETURN_NONE;
    // one allocation: sums, entry slots, ring slots, counts (8 bytes each), positions (4)
    const int64_t longs = 2 * (batch + 1) + entries + tokens + 4;
    const at::Tensor buf = at::empty({longs + (tokens + 1) / 2}, old_len->options().dtype(at::kLong));
    at::Tensor out[6];
    int64_t byte = 0;
    const auto next = [&](int64_t count, at::ScalarType type) {
        at::Tensor t = part(buf, type, byte, count);
        byte += count * (type == at::kInt ? 4 : 8);
        return t;
    };
    out[0] = next(batch + 1, at::kLong);
    out[1] = next(batch + 1, at::kLong);
    out[2] = next(entries, at::kLong);
    out[4] = next(tokens, at::kLong);
    out[5] = next(4, at::kLong);
    out[3] = next(tokens, at::kInt);
    const size_t need = abi.plan_bytes((int)batch);
    const at::Tensor ws = bytes_like(*old_len, need);
    void *st = stream_of(a.device);
    const auto longs_at = [&](int i) { return static_cast<long long *>(out[i].data_ptr()); };
    const int rc = call([&] {
        return abi.plan(ptr<int>(old_len), ptr<int>(new_len), (int)batch, (int)m, (int)page, (int)ring, ptr<int>(free_pages),
                        free_pages->size(0), static_cast<int *>(table->data_ptr()), (int)columns, longs_at(0), longs_at(1),
                        longs_at(2), entries, static_cast<int *>(out[3].data_ptr()), longs_at(4), tokens, longs_at(5),
                        need ? ws.data_ptr() : nullptr, need, st);
    });
    if (rc != CSA_OK) Py_RETURN_NONE;
    PyObject *tuple = PyTuple_New(6);
    if (!tuple) return nullptr;
    for (int i = 0; i < 6; ++i) PyTuple_SET_ITEM(tuple, i, THPVariable_Wrap(std::move(out[i])));
    return tuple;
    END_HANDLE_TH_ERRORS
}

// rows, slots, pool (bf16: 3 arguments) or codes, exps (4)
PyObject *paged_write(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const bool fp8 = n == 4;
    Args a(args, n, fp8 ? 4 : 3);
    const at::Tensor *rows = a.tensor(0, at::kBFloat16, 2), *slots = a.tensor(1, at::kLong, 1),
                     *pool = a.tensor(2, fp8 ? at::kByte : at::kBFloat16, -1),
                     *exps = fp8 ? a.tensor(3, at::kByte, -1) : nullptr;
    if (!a.ok || pool->dim() < 1) Py_RETURN_NONE;
    const int64_t d = pool->size(-1);
    if (d < 8 || d > 0x7fffffff || rows->size(1) != d || slots->size(0) != rows->size(0)) Py_RETURN_NONE;
    if (fp8) {
        if (exps->dim() != pool->dim() || exps->size(-1) != d / 128) Py_RETURN_NONE;
        for (int64_t i = 0; i + 1 < pool->dim(); ++i)
            if (exps->size(i) != pool->size(i)) Py_RETURN_NONE;
    }
    void *st = stream_of(a.device);
    const int rc = call([&] {
        const long long *at = ptr<long long>(slots);
        return fp8 ? abi.write_fp8(ptr<uint16_t>(rows), at, rows->size(0), (int)d, static_cast<uint8_t *>(pool->data_ptr()),
                                   static_cast<uint8_t *>(exps->data_ptr()), pool->numel() / d, st)
                   : abi.write(ptr<uint16_t>(rows), at, rows->size(0), (int)d, static_cast<uint16_t *>(pool->data_ptr()),
                               pool->numel() / d, st);
    });
    if (rc != CSA_OK) Py_RETURN_NONE;
    Py_RETURN_TRUE;
    END_HANDLE_TH_ERRORS
}

// q, pool, pool_exp or None, block_table, m, ring, ring_exp or None, q_pos, W, scale, eps, q_gain, n_shared, sinks, rope
PyObject *attend_paged(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 15);
    const bool fp8 = a.ok && args[2] != Py_None;
    const at::ScalarType type = fp8 ? at::kByte : at::kBFloat16;
    const at::Tensor *q = a.tensor(0, at::kBFloat16, 4), *pool = a.tensor(1, type, 3), *pool_e = a.optional(2, type, 3),
                     *table = a.tensor(3, at::kInt, 2), *ring = a.tensor(5, type, 3), *ring_e = a.optional(6, type, 3),
                     *pos = a.tensor(7, at::kInt, 2), *gain = a.optional(11, at::kFloat, 1),
                     *sinks = a.optional(13, at::kFloat, 1);
    const long long m = a.integer(4), W = a.integer(8), shared = a.integer(12);
    const double scale = a.real(9), eps = a.real(10);
    const at::Tensor *cos = nullptr, *sin = nullptr;
    if (a.ok && args[14] != Py_None) {
        if (!PyTuple_CheckExact(args[14]) || PyTuple_GET_SIZE(args[14]) != 2) Py_RETURN_NONE;
        cos = a.of(PyTuple_GET_ITEM(args[14], 0), at::kFloat, 2);
        sin = a.of(PyTuple_GET_ITEM(args[14], 1), at::kFloat, 2);
    }
    if (!a.ok) Py_RETURN_NONE;
    const int64_t batch = q->size(0), nq = q->size(1), H = q->size(2), D = q->size(3);
    for (const int64_t v : {batch, nq, H, D, pool->size(0), pool->size(1), table->size(1), ring->size(1)})
        if (v < 1 || v > 0x7fffffff) Py_RETURN_NONE;
    if (pool->size(2) != D || ring->size(2) != D || table->size(0) != batch || ring->size(0) != batch ||
        pos->size(0) != batch || pos->size(1) != nq || (gain && gain->size(0) != D) || (sinks && sinks->size(0) != H))
        Py_RETURN_NONE;
    if (cos && (cos->sizes() != sin->sizes() || cos->size(1) != 32 || D < 64)) Py_RETURN_NONE;
    if (fp8) {
        if (!ring_e) Py_RETURN_NONE;
        for (const auto &x : {std::make_pair(pool, pool_e), std::make_pair(ring, ring_e)})
            if (x.second->size(0) != x.first->size(0) || x.second->size(1) != x.first->size(1) || x.second->size(2) != D / 128)
                Py_RETURN_NONE;
    }
    const int page = (int)pool->size(1), columns = (int)table->size(1), ring_rows = (int)ring->size(1);
    const long long n_pages = pool->size(0), positions = cos ? cos->size(0) : 0;
    const size_t need = abi.attend_bytes((int)batch, (int)nq, (int)H, (int)D, page, columns, shared, ring_rows, (int)W, fp8,
                                         gain || cos || (float)scale < 0.f);
    at::Tensor out = at::empty(q->sizes(), q->options());
    const at::Tensor ws = bytes_like(*q, need);
    void *st = stream_of(a.device), *wp = need ? ws.data_ptr() : nullptr;
    const int rc = call([&] {
        uint16_t *o = static_cast<uint16_t *>(out.data_ptr());
        return fp8 ? abi.attend_fp8(ptr<uint16_t>(q), ptr<float>(gain), ptr<float>(sinks), ptr<float>(cos), ptr<float>(sin),
                                    positions, ptr<uint8_t>(pool), ptr<uint8_t>(pool_e), n_pages, page, ptr<int>(table), columns,
                                    shared, (int)m, ptr<uint8_t>(ring), ptr<uint8_t>(ring_e), ring_rows, (int)W, ptr<int>(pos),
                                    (int)batch, (int)nq, (int)H, (int)D, (float)scale, (float)eps, o, wp, need, st)
                   : abi.attend(ptr<uint16_t>(q), ptr<float>(gain), ptr<float>(sinks), ptr<float>(cos), ptr<float>(sin),
                                positions, ptr<uint16_t>(pool), n_pages, page, ptr<int>(table), columns, shared, (int)m,
                                ptr<uint16_t>(ring), ring_rows, (int)W, ptr<int>(pos), (int)batch, (int)nq, (int)H, (int)D,
                                (float)scale, (float)eps, o, wp, need, st);
    });
    if (rc != CSA_OK) Py_RETURN_NONE;
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}

PyMethodDef methods[] = {
    {"bind", bind, METH_O, nullptr},
    {"plan_pages", fast(plan_pages), METH_FASTCALL, nullptr},
    {"paged_write", fast(paged_write), METH_FASTCALL, nullptr},
    {"attend_paged", fast(attend_paged), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", CSA_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
