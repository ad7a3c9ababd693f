// The calls of the attention layers and the acceptance for Python without its
// cost: of the 8 to 11 us that api.py spends around a library call, most are
// some fifty queries of tensors from Python and the allocations.  Back to back
// on a GB300's host an append takes 4.8 us so and 11.9 without, an attention
// 8.6 and 18.2, log probabilities 6.3 and 15.6.
//
// Each function takes the address of the library's packed entry point and
// api.py's arguments in order.  It answers None, having done nothing, where
// anything is not plainly as it should be (api.py then finds out what, and
// says so), the library's status where that is not 0, and the outputs.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "kda.h"

namespace {

using at::Tensor;

struct NotPlain {};  // thrown where api.py has to look

void need(bool ok) {
    if (!ok) throw NotPlain{};
}

// The library launches on the current device; where the tensors are on another
// GPU, api.py switches to it.
void need_current(c10::Device device) {
    need(device.is_cuda() && device.index() == c10::cuda::current_device());
}

const Tensor &tensor(PyObject *o) {
    need(THPVariable_Check(o));
    return THPVariable_Unpack(o);
}

// A tensor of this type on this GPU.
const Tensor &tensor(PyObject *o, at::ScalarType type, c10::Device device) {
    const Tensor &t = tensor(o);
    need(t.scalar_type() == type && t.device() == device && t.layout() == at::kStrided);
    return t;
}

int32_t integer(PyObject *o) {
    need(PyLong_CheckExact(o));
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
    need(overflow == 0 && v >= INT_MIN && v <= INT_MAX);
    return (int32_t)v;
}

int32_t narrow(int64_t v) {
    need(v >= 0 && v <= INT_MAX);
    return (int32_t)v;
}

int32_t dtype_code(at::ScalarType t) {
    need(t == at::kBFloat16 || t == at::kHalf || t == at::kFloat);
    return t == at::kBFloat16 ? KDA_DTYPE_BF16 : t == at::kHalf ? KDA_DTYPE_FP16 : KDA_DTYPE_FP32;
}

// Both caches: their type, shape and strides.  The stride of a dimension of one
// element says nothing and may be anything; a head's channels stand for it.
void set_cache(kda_cache_config &c, int32_t &block_size, const Tensor &keys, const Tensor &values) {
    need(keys.dim() == 4 && keys.stride(3) == 1 && values.dim() == 4 && values.stride(3) == 1 &&
         values.sizes() == keys.sizes() && keys.scalar_type() != at::kFloat);
    int64_t strides[3];
    for (int i = 0; i < 3; ++i) {
        const bool one = keys.size(i) == 1;
        need(one || values.stride(i) == keys.stride(i));
        strides[i] = one ? keys.size(3) : keys.stride(i);
    }
    c.dtype = dtype_code(keys.scalar_type());
    c.num_blocks = narrow(keys.size(0));
    block_size = narrow(keys.size(1));
    c.kv_heads = narrow(keys.size(2));
    c.head_dim = narrow(keys.size(3));
    c.stride_block = strides[0];
    c.stride_token = strides[1];
    c.stride_head = strides[2];
}

// A [T, heads, dim] activation, heads and channels packed: its token stride.
int64_t token_stride(const Tensor &t, int64_t dim) {
    need(t.dim() == 3 && t.size(2) == dim && t.stride(2) == 1 &&
         (t.stride(1) == dim || t.size(1) <= 1));
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * dim;
}

// The rows' side of a call.
int32_t set_rows(kda_align &a, int32_t block_size, const Tensor &cu, const Tensor &table,
                 const Tensor &computed, PyObject *requests, c10::Device device) {
    const int32_t rows = narrow(cu.numel() - 1);
    need(cu.is_contiguous() && table.dim() == 2 && (table.stride(1) == 1 || table.size(1) <= 1) &&
         computed.is_contiguous() && computed.numel() >= table.size(0));
    a = kda_align{};
    a.block_table = table.const_data_ptr<int32_t>();
    a.block_table_stride = table.size(0) > 1 ? table.stride(0) : table.size(1);
    a.block_table_width = narrow(table.size(1));
    a.block_size = block_size;
    a.num_requests = narrow(table.size(0));
    a.num_computed = computed.const_data_ptr<int32_t>();
    if (requests != Py_None) {
        const Tensor &r = tensor(requests, at::kInt, device);
        need(r.is_contiguous() && r.numel() >= rows);
        a.request_indices = r.const_data_ptr<int32_t>();
    } else {
        need(rows <= a.num_requests);
    }
    return rows;
}

int32_t *error_address(PyObject *o, c10::Device device) {
    if (o == Py_None) return nullptr;
    const Tensor &e = tensor(o, at::kInt, device);
    need(e.numel() >= 1);
    return e.data_ptr<int32_t>();
}

// Other threads run Python meanwhile: an allocation or a launch may wait for
// the GPU, and what runs there may wait for a host function in Python.
struct Unlocked {
    PyThreadState *const state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

Tensor allocate(at::IntArrayRef shape, at::ScalarType type, c10::Device device) {
    const Unlocked unlocked;
    return at::empty(shape, at::dtype(type).device(device));
}

// The output that was given, checked, or a new one.
Tensor output(PyObject *given, at::IntArrayRef shape, at::ScalarType type, c10::Device device) {
    if (given == Py_None) return allocate(shape, type, device);
    const Tensor &t = tensor(given, type, device);
    need(t.sizes() == shape && t.is_contiguous());
    return t;
}

// A contiguous tensor in the memory of `all`, from its element `at` on, of a
// type of the same size: 0.1 us, where one of its own takes 0.6.
Tensor part(const Tensor &all, int64_t at, at::IntArrayRef shape, at::ScalarType type) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        c10::Storage(all.storage()), all.key_set(), c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    return t;
}

template <typename Args>
int call(PyObject *address, const Args &args) {
    const auto function = reinterpret_cast<int (*)(const Args *)>(PyLong_AsVoidPtr(address));
    const Unlocked unlocked;
    return function(&args);
}

template <typename Body>
PyObject *guarded(Body body) {
    try {
        return body();
    } catch (...) {  // also what torch throws: api.py meets it again
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// address, q, k, v, key_cache, value_cache, cu_seqlens, block_table,
// num_computed, inv_freq, interleaved, q_out, request_indices, error_word
PyObject *append(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 14);
        const Tensor &keys = tensor(o[4]);
        const c10::Device device = keys.device();
        need_current(device);
        const at::ScalarType type = keys.scalar_type();
        const Tensor &k = tensor(o[2], type, device), &v = tensor(o[3], type, device);
        const Tensor &values = tensor(o[5], type, device);
        const Tensor &cu = tensor(o[6], at::kInt, device), &table = tensor(o[7], at::kInt, device);
        const Tensor &computed = tensor(o[8], at::kInt, device);
        kda_append_args a{};
        kda_cache_config &c = a.config;
        int32_t block_size;
        set_cache(c, block_size, keys, values);
        a.B = set_rows(a.align, block_size, cu, table, computed, o[12], device);
        c.stride_k_t = token_stride(k, c.head_dim);
        c.stride_v_t = token_stride(v, c.head_dim);
        need(k.size(1) == c.kv_heads && v.size(1) == c.kv_heads && v.size(0) == k.size(0));
        a.num_tokens = narrow(k.size(0));
        c.q_heads = c.kv_heads;
        c.window = 1;
        c.scale = 1.0f;
        c.stride_q_t = 8;
        Tensor rotated;
        if (o[1] != Py_None) {
            const Tensor &q = tensor(o[1], type, device);
            c.stride_q_t = token_stride(q, c.head_dim);
            c.q_heads = narrow(q.size(1));
            need(q.size(0) == k.size(0) && c.kv_heads > 0 && c.q_heads > 0 &&
                 c.q_heads % c.kv_heads == 0);
            rotated = output(o[11], q.sizes(), type, device);
            a.q = q.const_data_ptr();
            a.q_out = rotated.data_ptr();
        } else {
            need(o[11] == Py_None);
        }
        if (o[9] != Py_None) {
            const Tensor &f = tensor(o[9], at::kDouble, device);
            need(f.dim() == 1 && f.is_contiguous());
            c.rotary_dim = narrow(2 * f.numel());
            a.inv_freq = f.const_data_ptr<double>();
        }
        const int interleaved = PyObject_IsTrue(o[10]);
        need(interleaved >= 0);  // no truth value: it raises again in api.py
        c.interleaved = interleaved;
        a.k = k.const_data_ptr();
        a.v = v.const_data_ptr();
        a.key_cache = keys.data_ptr();
        a.value_cache = values.data_ptr();
        a.cu_seqlens = cu.const_data_ptr<int32_t>();
        a.error_word = error_address(o[13], device);
        a.stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
        if (const int status = call(o[0], a)) return PyLong_FromLong(status);
        PyObject *result = PyTuple_New(1);
        if (result == nullptr) return nullptr;
        if (o[1] == Py_None)
            PyTuple_SET_ITEM(result, 0, Py_NewRef(Py_None));
        else
            PyTuple_SET_ITEM(result, 0,
                             o[11] != Py_None ? Py_NewRef(o[11]) : THPVariable_Wrap(rotated));
        return result;
    });
}

// address, q, key_cache, value_cache, cu_seqlens, block_table, num_computed,
// workspace, window, scale, left_window, request_indices, out, lse, error_word
PyObject *attend(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 15);
        const Tensor &keys = tensor(o[2]);
        const c10::Device device = keys.device();
        need_current(device);
        const at::ScalarType type = keys.scalar_type();
        const Tensor &q = tensor(o[1], type, device), &values = tensor(o[3], type, device);
        const Tensor &cu = tensor(o[4], at::kInt, device), &table = tensor(o[5], at::kInt, device);
        const Tensor &computed = tensor(o[6], at::kInt, device);
        const Tensor &work = tensor(o[7], at::kByte, device);
        kda_attention_args a{};
        kda_cache_config &c = a.config;
        int32_t block_size;
        set_cache(c, block_size, keys, values);
        a.B = set_rows(a.align, block_size, cu, table, computed, o[11], device);
        c.stride_q_t = token_stride(q, c.head_dim);
        c.stride_k_t = c.stride_v_t = 8;
        c.q_heads = narrow(q.size(1));
        need(c.kv_heads > 0 && c.q_heads > 0 && c.q_heads % c.kv_heads == 0 && q.size(0) > 0 &&
             work.is_contiguous());
        a.num_tokens = narrow(q.size(0));
        c.window = o[8] != Py_None
                       ? integer(o[8])
                       : std::min(KDA_MAX_WINDOW,
                                  std::max(1, KDA_MAX_QUERY_ROWS / (c.q_heads / c.kv_heads)));
        c.left_window = integer(o[10]);
        need(o[9] == Py_None || PyFloat_CheckExact(o[9]));
        c.scale = (float)(o[9] == Py_None ? 1.0 / std::sqrt((double)c.head_dim)
                                          : PyFloat_AS_DOUBLE(o[9]));
        const Tensor out = output(o[12], q.sizes(), type, device);
        const Tensor lse = output(o[13], {q.size(0), q.size(1)}, at::kFloat, device);
        a.q = q.const_data_ptr();
        a.key_cache = keys.const_data_ptr();
        a.value_cache = values.const_data_ptr();
        a.cu_seqlens = cu.const_data_ptr<int32_t>();
        a.workspace = work.data_ptr();
        a.workspace_bytes = (uint64_t)work.numel();
        a.out = out.data_ptr();
        a.lse = lse.data_ptr<float>();
        a.error_word = error_address(o[14], device);
        a.stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
        if (const int status = call(o[0], a)) return PyLong_FromLong(status);
        PyObject *result = PyTuple_New(2);
        if (result == nullptr) return nullptr;
        PyTuple_SET_ITEM(result, 0, o[12] != Py_None ? Py_NewRef(o[12]) : THPVariable_Wrap(out));
        PyTuple_SET_ITEM(result, 1, o[13] != Py_None ? Py_NewRef(o[13]) : THPVariable_Wrap(lse));
        return result;
    });
}

// address, logits, tokens, num_top, error_word
PyObject *logprobs(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 5);
        const Tensor &x = tensor(o[1]);
        const c10::Device device = x.device();
        need_current(device);
        need(x.dim() == 2 && (x.stride(1) == 1 || x.size(1) <= 1) &&
             x.layout() == at::kStrided);
        const Tensor &tokens = tensor(o[2], at::kInt, device);
        need(tokens.dim() == 1 && tokens.numel() == x.size(0) && tokens.is_contiguous());
        kda_logprobs_args a{};
        a.dtype = dtype_code(x.scalar_type());
        a.rows = narrow(x.size(0));
        a.vocab = narrow(x.size(1));
        a.num_top = integer(o[3]);
        need(a.num_top >= 0 && a.num_top <= KDA_MAX_TOP);
        const int64_t rows = a.rows, top = a.num_top;
        const Tensor all = allocate({rows * (3 + 2 * top)}, at::kFloat, device);
        const Tensor outputs[5] = {part(all, 0, {rows}, at::kFloat),
                                   part(all, rows, {rows}, at::kFloat),
                                   part(all, 2 * rows, {rows}, at::kFloat),
                                   part(all, 3 * rows, {rows, top}, at::kFloat),
                                   part(all, (3 + top) * rows, {rows, top}, at::kInt)};
        a.logits = x.const_data_ptr();
        a.stride_row = x.stride(0);
        a.tokens = tokens.const_data_ptr<int32_t>();
        a.logprob = outputs[0].data_ptr<float>();
        a.entropy = outputs[1].data_ptr<float>();
        a.lse_out = outputs[2].data_ptr<float>();
        a.top_logprob = outputs[3].data_ptr<float>();
        a.top_index = outputs[4].data_ptr<int32_t>();
        a.error_word = error_address(o[4], device);
        a.stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
        if (const int status = call(o[0], a)) return PyLong_FromLong(status);
        PyObject *result = PyTuple_New(5);
        if (result == nullptr) return nullptr;
        for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(result, i, THPVariable_Wrap(outputs[i]));
        return result;
    });
}

template <PyObject *(*kFunction)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kFunction)),
            METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<append>("append"), method<attend>("attend"),
                         method<logprobs>("logprobs"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// What this was built for: api.py uses it only where its own structures have the
// same sizes and PyTorch, whose tensors are laid out in here, is the same.
PyMODINIT_FUNC PyInit__binding() {
    PyObject *m = PyModule_Create(&module);
    if (m == nullptr) return nullptr;
    PyObject *sizes = Py_BuildValue("(nnn)", (Py_ssize_t)sizeof(kda_append_args),
                                    (Py_ssize_t)sizeof(kda_attention_args),
                                    (Py_ssize_t)sizeof(kda_logprobs_args));
    if (sizes == nullptr || PyModule_AddObject(m, "argument_sizes", sizes) != 0 ||
        PyModule_AddStringConstant(m, "torch_version", KDA_TORCH_VERSION) != 0) {
        Py_XDECREF(m);
        return nullptr;
    }
    return m;
}
